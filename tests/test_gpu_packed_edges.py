"""Packed attention at the ends of what its inputs may hold (GB300)."""

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
@pytest.mark.parametrize("nh,nkv,d,n", [(4, 2, 64, 128), (3, 3, 64, 256), (2, 1, 128, 256), (3, 1, 96, 130), (5, 5, 128, 128),
                                        (4, 2, 160, 64), (3, 3, 160, 200)])
def test_first_keys_of_no_weight(nh, nkv, d, n, fill):
    cu, T = [0, 37, 457, 462], 462
    g = torch.Generator().manual_seed(n + d)
    q = (torch.randn(T, nh, d, generator=g).abs() + 0.1).to(BF)  # every product with `fill` has its sign
    k, v = (torch.randn(T, nkv, d, generator=g).to(BF) for _ in range(2))
    do = torch.randn(T, nh, d, generator=g).to(BF)
    k[cu[1]:cu[1] + n] = fill
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O, lse = binding.tp_attn_packed_forward(q.cuda(), k.cuda(), v.cuda(), cud)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    rows = torch.ones(T, dtype=torch.bool)
    rows[cu[1]:cu[1] + n] = False  # these see no other keys
    Or, lr, A = ref.attention(q, k, v, cu, d ** -0.5)
    Or, lr, A = Or[rows], lr[:, rows], A[rows]
    assert torch.isfinite(Or).all() and torch.isfinite(lr).all()
    # P rounded to bf16, O rounded to bf16, exponents of sums of d <= 160 terms in fp32:
    # d 2^-24 times sum |q k| scale log2(e) < 24 is below 2^-12
    tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (A + Or.abs()) + 2.0 ** -11 * A
    assert ((O.double().cpu()[rows] - Or).abs() <= tol).all()
    assert ((lse.double().cpu()[:, rows] - lr).abs() <= 2.0 ** -11 + 2.0 ** -21 * lr.abs()).all()
    if fill == -math.inf:
        # rows without a finite score have no softmax
        assert torch.isnan(O.cpu()[~rows].float()).all() and (lse.cpu()[:, ~rows] == -math.inf).all()
        return
    # dQ of the other rows (dK and dV sum over all of them)
    Oall, lall, _ = ref.attention(q, k, v, cu, d ** -0.5)
    o, l32 = Oall.to(BF), lall.float()
    dQ, _, _ = binding.tp_attn_packed_backward(q.cuda(), k.cuda(), v.cuda(), o.cuda(), l32.cuda(), do.cuda(), cud)
    (want, _, _), (t, _, _) = ref.attention_backward(q, k, v, o, l32, do, cu, d ** -0.5)
    assert torch.isfinite(want[rows]).all()
    assert ((dQ.double().cpu() - want).abs() <= t)[rows].all()


def test_bad_offsets_leave_an_earlier_timeout():
    x = torch.zeros(100, 2, 64, dtype=BF, device="cuda")
    bad = torch.tensor([0, 50, 40, 90], dtype=torch.int32, device="cuda")
    assert binding.device_status() == binding.TPMLP_OK
    # a wait that gives up after 2 ms, whose status is not read
    assert binding.lib().tpmlp_selftest_bounded_wait(2000, torch.cuda.current_stream().cuda_stream) == binding.TPMLP_OK
    binding.tp_attn_packed_forward(x, x, x, bad)
    assert binding.device_status() == binding.TPMLP_ERR_DEVICE_TIMEOUT
    binding.tp_attn_packed_forward(x, x, x, bad)
    assert binding.device_status() == binding.TPMLP_ERR_SHAPE
    assert binding.device_status() == binding.TPMLP_OK


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# groups of 5, 7 and 13 heads in 2 and 6 parts, of unequal size
@pytest.mark.parametrize("nb,nh,nkv,d", [(20, 40, 8, 64), (40, 21, 3, 128), (40, 13, 1, 160), (40, 13, 1, 96)])
def test_groups_dealt_to_unequal_parts(nb, nh, nkv, d):
    g = torch.Generator().manual_seed(nh + d)
    lens = [int(n) for n in torch.randint(0, 130, (nb,), generator=g)]
    cu = _cu(lens)
    T = cu[-1] + 3
    q, k, v, do = (torch.randn(T, n, d, generator=g).to(BF) for n in (nh, nkv, nkv, nh))
    Or, lr, _ = ref.attention(q, k, v, cu, d ** -0.5)
    o, l32 = Or.to(BF), lr.float()
    gpu = [x.cuda() for x in (q, k, v, o, l32, do)]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = [torch.full((T, n, d), 7.0, dtype=BF, device="cuda") for n in (nh, nkv, nkv)]
    got = binding.tp_attn_packed_backward(*gpu, cud, dQ=out[0], dK=out[1], dV=out[2])
    assert binding.last_launch_count() == 4  # delta and plan, dQ, dK and dV, parts
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    want, tol = ref.attention_backward(q, k, v, o, l32, do, cu, d ** -0.5)
    for name, x, w, t in zip(("dQ", "dK", "dV"), got, want, tol):
        err = (x.double().cpu() - w).abs()[:cu[-1]]
        assert (err <= t[:cu[-1]]).all(), (name, (err - t[:cu[-1]]).max())
        assert (x[cu[-1]:] == 7.0).all()
    again = binding.tp_attn_packed_backward(*gpu, cud)
    assert all(torch.equal(a[:cu[-1]], b[:cu[-1]]) for a, b in zip(got, again))


def test_scratch_of_the_largest_batch_serves_the_smaller_ones():
    nh, nkv, d = 16, 4, 160
    need = binding.lib().tp_attn_packed_backward_workspace_bytes(23, 6007, nh, nkv, d)
    room = torch.full((need + 4096,), 90, dtype=torch.uint8, device="cuda")
    for nb, T in ((23, 6007), (10, 6007), (10, 5000), (1, 3000), (2, 1)):
        g = torch.Generator(device="cuda").manual_seed(T)
        q, k, v, do = (torch.randn(T, n, d, generator=g, device="cuda").to(BF) for n in (nh, nkv, nkv, nh))
        cu = (torch.arange(nb + 1, device="cuda") * T // nb).int()
        O, lse = binding.tp_attn_packed_forward(q, k, v, cu, workspace=room[:need])
        a = binding.tp_attn_packed_backward(q, k, v, O, lse, do, cu, workspace=room[:need])
        b = binding.tp_attn_packed_backward(q, k, v, O, lse, do, cu)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert (room[need:] == 90).all() and binding.device_status() == 0
    with pytest.raises(binding.TpMlpError):
        binding.tp_attn_packed_backward(q, k, v, O, lse, do, cu, workspace=room[:64])


def test_a_batch_without_tokens():
    e = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    O, lse = binding.tp_attn_packed_forward(e, e[:, :2], e[:, :2], cu)
    dQ, dK, dV = binding.tp_attn_packed_backward(e, e[:, :2], e[:, :2], O, lse, e, cu)
    assert dQ.shape == (0, 4, 64) and dK.shape == dV.shape == (0, 2, 64)
