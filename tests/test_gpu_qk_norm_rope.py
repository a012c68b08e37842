"""Norms of queries and keys with the rotation, against their 64-bit form (GB300)."""

import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32

CASES = [
    # T, nh, nkv, d, rot, type, theta, first position
    (1, 1, 1, 32, 32, BF, 1e4, 0),
    (1, 32, 8, 128, 128, BF, 1e4, 131071),
    (7, 3, 1, 64, 64, HF, 1e4, 0),
    (33, 5, 5, 96, 96, FP, 5e5, 1 << 20),
    (129, 20, 5, 96, 64, HF, 1e4, 4000),
    (50, 2, 2, 160, 80, BF, 1e4, -60),
    (65, 4, 2, 256, 256, FP, 1e6, 2**31 - 66),
    (300, 1, 1, 32, 16, FP, 0.5, 0),
    (40, 7, 2, 48, 0, BF, 1e4, 0),
    (1000, 6, 2, 128, 128, FP, 1e4, 65536),
    (513, 16, 16, 64, 32, BF, 1e4, -2**31),
    (5, 1, 1, 240, 224, HF, 1e4, 3),
]


def _make(T, nh, nkv, d, dt, first, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    size = torch.exp(torch.randn(T, 1, 1, generator=g)).to(dt)
    q, k = r(T, nh, d) * size, r(T, nkv, d)
    dq, dk = r(T, nh, d), r(T, nkv, d)
    gq, gk = (1 + 0.2 * torch.randn(d, generator=g)).to(dt), (1 + 0.2 * torch.randn(d, generator=g)).to(dt)
    pos = (first + torch.arange(T, dtype=torch.int64)).to(torch.int32)[torch.randperm(T, generator=g)]
    return q, k, dq, dk, gq, gk, pos


def _part(x, y):
    """x and y as parts of one matrix of rows with 8 values more, on the GPU."""
    T, nh, d = x.shape
    n = nh + y.shape[1]
    rows = torch.full((T, n * d + 8), 7.0, dtype=x.dtype, device="cuda")
    a, b = rows[:, :nh * d].unflatten(1, (nh, d)), rows[:, nh * d:n * d].unflatten(1, (n - nh, d))
    a.copy_(x)
    b.copy_(y)
    return a, b, rows


@pytest.mark.parametrize("T,nh,nkv,d,rot,dt,theta,first", CASES)
def test_forward_and_backward(T, nh, nkv, d, rot, dt, theta, first):
    q, k, dq, dk, gq, gk, pos = _make(T, nh, nkv, d, dt, first, seed=T + d)
    qs, ks, _ = _part(q, k)
    dqs, dks, _ = _part(dq, dk)
    eps = 1e-5
    gpu = [x.cuda() for x in (gq, gk, pos)]
    Qo, Ko, rows = _part(torch.zeros_like(q), torch.zeros_like(k))
    _, _, rstd = binding.tp_qk_norm_rope_forward(qs, ks, *gpu, rot=rot, theta=theta, eps=eps, Qo=Qo, Ko=Ko)
    half = ref.HALF[dt]
    # an fp32 angle is off by 2^-24 of at most 1/8 turn and its sine by two steps:
    # 2^-21; the mean of d <= 256 squares by d 2^-25 halved by the root; six products
    wide = 2.0 ** -21 + d * 2.0 ** -25 + 6 * 2.0 ** -24
    # 64-bit angles of the reference itself: positions up to 2^31, 2^-52 relative
    wide += 2.0 ** 31 * 2.0 ** -52
    want_r = []
    for got, x, gamma in ((Qo, q, gq), (Ko, k, gk)):
        y, r, size = ref.qk_forward(x, gamma, pos, rot, theta, eps)
        want_r.append(r)
        assert ((got.double().cpu() - y).abs() <= half * (y.abs() + 2.0 ** -10 * size) + wide * size
                + (2.0 ** -25 if dt is HF else 0.0)).all()
    want_r = torch.cat(want_r, 1)
    assert ((rstd.double().cpu() - want_r).abs() <= (2.0 ** -23 + d * 2.0 ** -25) * want_r).all()
    assert (rows[:, (nh + nkv) * d:] == 7.0).all()

    r32 = want_r.float()
    dQ, dK, rows = _part(torch.zeros_like(q), torch.zeros_like(k))
    got = binding.tp_qk_norm_rope_backward(dqs, dks, qs, ks, *gpu, r32.cuda(), rot=rot, theta=theta, dQ=dQ, dK=dK)
    for x, dy, gamma, r, gx, gg in ((q, dq, gq, r32[:, :nh], got[0], got[2]), (k, dk, gk, r32[:, nh:], got[1], got[3])):
        dx, dg, dx_size, dg_size = ref.qk_backward(dy, x, gamma, pos, r, rot, theta)
        assert ((gx.double().cpu() - dx).abs() <= half * (dx.abs() + 2.0 ** -10 * dx_size) + 2 * wide * dx_size
                + (2.0 ** -25 if dt is HF else 0.0)).all()
        # sums of T * heads terms: at most 2^5 run in one thread's chain here, then the
        # CTAs' parts; 2^-18 covers chains of 64
        assert ((gg.double().cpu() - dg).abs() <= (wide + 2.0 ** -18) * dg_size).all()
    assert (rows[:, (nh + nkv) * d:] == 7.0).all()


def test_zero_rows_and_special_values():
    T, d = 9, 128
    q = torch.zeros(T, 2, d, dtype=BF)
    k = torch.randn(T, 1, d).to(BF)
    k[3, 0, 5] = math.nan
    k[4, 0, 7] = math.inf
    one, pos = torch.ones(d, dtype=BF), torch.arange(T, dtype=torch.int32)
    Qo, Ko, rstd = binding.tp_qk_norm_rope_forward(q.cuda(), k.cuda(), one.cuda(), one.cuda(), pos.cuda())
    assert (Qo == 0).all() and torch.isfinite(rstd[:, :2]).all()  # eps keeps a row of zeros finite
    fine = [t for t in range(T) if t not in (3, 4)]
    assert torch.isfinite(Ko[fine].float()).all()
    assert torch.isnan(Ko[3].float()).all() and not torch.isfinite(Ko[4, 0, 7].float())
    # position 0 turns nothing
    y, _, _ = ref.qk_forward(k[:1], one, pos[:1], d, 1e4, 1e-5)
    assert ((Ko[:1].double().cpu() - y).abs() <= 2.0 ** -7 * y.abs()).all()


def test_a_turn_and_its_inverse():
    # fp32 at the far ends of the positions: R(-p) R(p) x = x
    T, d = 64, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 2, d, generator=g)
    x = x / (x * x).mean(-1, keepdim=True).sqrt()
    pos = torch.randint(-2**31, 2**31 - 1, (T,), generator=g).to(torch.int32).cuda()
    one = torch.ones(d, device="cuda")
    Qo, Ko, rstd = binding.tp_qk_norm_rope_forward(x.cuda(), x[:, :1].cuda(), one, one, pos, eps=1e-30)
    # dy = y: g = R(-p) R(p) xhat, so dgamma = sum xhat^2
    _, _, dgq, _ = binding.tp_qk_norm_rope_backward(Qo, Ko, x.cuda(), x[:, :1].cuda(), one, one, pos, rstd)
    want = (x.double() ** 2).sum((0, 1))
    assert ((dgq.double().cpu() - want).abs() <= 2.0 ** -18 * (x.double() ** 2).sum() / d * 2).all()


def test_repeats_streams_graph_and_empty():
    q, k, dq, dk, gq, gk, pos = (x.cuda() for x in _make(700, 8, 2, 128, BF, 0, seed=4))
    a = binding.tp_qk_norm_rope_forward(q, k, gq, gk, pos)
    first = binding.tp_qk_norm_rope_backward(dq, dk, q, k, gq, gk, pos, a[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = binding.tp_qk_norm_rope_forward(q, k, gq, gk, pos, stream=s)
    again = binding.tp_qk_norm_rope_backward(dq, dk, q, k, gq, gk, pos, b[2], stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a + first, b + again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = binding.tp_qk_norm_rope_forward(q, k, gq, gk, pos)
        third = binding.tp_qk_norm_rope_backward(dq, dk, q, k, gq, gk, pos, c[2])
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(a + first, c + third))
    e = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    g64 = torch.ones(64, dtype=BF, device="cuda")
    p0 = torch.empty(0, dtype=torch.int32, device="cuda")
    Qo, Ko, rstd = binding.tp_qk_norm_rope_forward(e, e, g64, g64, p0)
    assert Qo.shape == (0, 4, 64) and rstd.shape == (0, 8)
    _, _, dgq, dgk = binding.tp_qk_norm_rope_backward(e, e, e, e, g64, g64, p0, rstd,
                                                      dgamma_q=torch.ones(64, device="cuda"))
    assert (dgq == 0).all() and (dgk == 0).all()
    with pytest.raises(binding.TpMlpError):
        binding.tp_qk_norm_rope_forward(q, k, gq, gk, pos, rot=24)
    with pytest.raises(ValueError, match="gamma_q"):
        binding.tp_qk_norm_rope_forward(q, k, gq.float(), gk, pos)
    with pytest.raises(ValueError, match="positions"):
        binding.tp_qk_norm_rope_forward(q, k, gq, gk, pos.long())


def test_offsets_past_32_bits():
    # token 2^24 and more of 128 values each, two heads apart in one matrix
    T, d = (1 << 24) + 40, 128
    q = torch.zeros(T, 1, d, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(6)
    tail = torch.randn(64, 1, d, generator=g).to(BF)
    q[T - 64:] = tail.cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    one = torch.ones(d, dtype=BF, device="cuda")
    Qo, Ko, _ = binding.tp_qk_norm_rope_forward(q, q, one, one, pos)
    y, _, size = ref.qk_forward(tail, one.cpu(), pos[T - 64:].cpu(), d, 1e4, 1e-5)
    for o in (Qo, Ko):
        assert ((o[T - 64:].double().cpu() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -17 * size).all()
        assert (o[:T - 64] == 0).all()
