"""Packed attention, norms and rotation of queries and keys, gradient clipping on
a host without a GPU: the 64-bit forms against differences, refusals, scratch."""

import ctypes
import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding, build
from tests import packed_reference as ref

P = ctypes.c_void_p(0x10000)
Q8 = ctypes.c_void_p(0x10008)  # 8-byte aligned only
O2 = ctypes.c_void_p(0x10002)
N = None
S, NU, AL, WS, OK = (binding.TPMLP_ERR_SHAPE, binding.TPMLP_ERR_NULL, binding.TPMLP_ERR_ALIGN,
                     binding.TPMLP_ERR_WORKSPACE, binding.TPMLP_OK)
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def _differences(f, x, eps=1e-6):
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        at = flat[i].item()
        flat[i] = at + eps
        up = f()
        flat[i] = at - eps
        out[i] = (up - f()) / (2 * eps)
        flat[i] = at
    return g


def test_attention_gradients_are_differences():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    cu, scale = [1, 4, 4, 5, 8], 0.7
    q, k, v, do = r(9, 4, 3), r(9, 2, 3), r(9, 2, 3), r(9, 4, 3)
    loss = lambda: float((ref.attention(q, k, v, cu, scale)[0][1:8] * do[1:8]).sum())  # noqa: E731
    o, lse, _ = ref.attention(q, k, v, cu, scale)
    grads, _ = ref.attention_backward(q, k, v, o, lse, do, cu, scale)
    for x, g in zip((q, k, v), grads):
        assert torch.allclose(_differences(loss, x), g, atol=1e-7)


@pytest.mark.parametrize("rot", [0, 4, 6])
def test_qk_gradients_are_differences(rot):
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, gamma, dy = r(4, 2, 6), r(6), r(4, 2, 6)
    pos = torch.tensor([0, 1, 77, -5])
    y = lambda: ref.qk_forward(x, gamma, pos, rot, 100.0, 1e-3)  # noqa: E731
    loss = lambda: float((y()[0] * dy).sum())  # noqa: E731
    dx, dgamma, _, _ = ref.qk_backward(dy, x, gamma, pos, y()[1], rot, 100.0)
    assert torch.allclose(_differences(loss, x), dx, atol=1e-7)
    assert torch.allclose(_differences(loss, gamma), dgamma, atol=1e-7)


def test_attention_refusals(L):
    big = 1 << 40

    def fwd(q=P, lq=512, k=P, lk=256, cu=P, nb=2, T=40, nh=8, nkv=4, d=64, sc=0.125, o=P, lse=P, ws=P, n=big):
        return L.tp_attn_packed_forward(q, lq, k, lk, P, 256, cu, nb, T, nh, nkv, d, sc, o, lse, ws, n, N)

    def bwd(do=P, lq=512, dq=P, ldq=512, dk=P, ldk=256, nb=2, T=40, nh=8, nkv=4, d=64, ws=P, n=big):
        return L.tp_attn_packed_backward(P, lq, P, 256, P, 256, P, P, do, P, nb, T, nh, nkv, d, 0.125, dq, ldq, dk,
                                         ldk, P, 256, ws, n, N)

    for kw in (dict(nb=-1), dict(T=-1), dict(nh=0), dict(nkv=0), dict(nkv=3), dict(d=80), dict(d=0), dict(sc=0.0),
               dict(sc=-1.0), dict(sc=NAN), dict(sc=INF), dict(sc=2.5e38), dict(lq=504), dict(lq=516), dict(lk=255), dict(lk=-256),
               dict(T=(1 << 30) + 1), dict(nb=(1 << 30) + 1), dict(nb=1 << 30)):
        assert fwd(**kw) == S, kw
    for kw in (dict(q=N), dict(k=N), dict(cu=N), dict(o=N), dict(lse=N)):
        assert fwd(**kw) == NU, kw
    for kw in (dict(q=Q8), dict(k=Q8), dict(o=Q8), dict(lse=Q8), dict(ws=Q8), dict(cu=O2)):
        assert fwd(**kw) == AL, kw
    need = L.tp_attn_packed_forward_workspace_bytes(2, 40, 8, 4, 64)
    assert fwd(ws=N) == WS and fwd(n=need - 1) == WS
    assert fwd(T=0, q=N, k=N, cu=N, o=N, lse=N, ws=N) == OK
    assert fwd(nb=0, q=N, k=N, cu=N, o=N, lse=N, ws=N) == OK
    for kw in (dict(T=-1), dict(nkv=5), dict(d=72), dict(ldq=511), dict(ldk=252), dict(lq=511)):
        assert bwd(**kw) == S, kw
    for kw in (dict(do=N), dict(dq=N), dict(dk=N)):
        assert bwd(**kw) == NU, kw
    for kw in (dict(do=Q8), dict(dq=Q8), dict(dk=Q8), dict(ws=Q8)):
        assert bwd(**kw) == AL, kw
    need = L.tp_attn_packed_backward_workspace_bytes(2, 40, 8, 4, 64)
    assert bwd(ws=N) == WS and bwd(n=need - 1) == WS
    assert bwd(T=0, do=N, dq=N, ws=N) == OK


def test_qk_refusals(L):
    def fwd(q=P, lq=512, lk=256, gq=P, pos=P, T=4, nh=4, nkv=2, d=128, rot=128, th=1e4, eps=1e-5, dt=0, qo=P, lqo=512,
            rstd=P):
        return L.tp_qk_norm_rope_forward(q, lq, P, lk, gq, P, pos, T, nh, nkv, d, rot, th, eps, dt, qo, lqo, P, 256,
                                         rstd, N)

    def bwd(dy=P, ldy=512, T=4, d=128, rot=64, th=1e4, dt=0, dq=P, ldq=512, dg=P, part=P):
        return L.tp_qk_norm_rope_backward(dy, ldy, P, 256, P, 512, P, 256, P, P, P, P, T, 4, 2, d, rot, th, dt, dq,
                                          ldq, P, 256, dg, P, part, N)

    for kw in (dict(T=-1), dict(nh=0), dict(nkv=0), dict(d=120, rot=64), dict(d=16, rot=16), dict(d=272), dict(rot=136),
               dict(rot=8), dict(rot=-16), dict(th=0.0), dict(th=NAN), dict(th=INF), dict(eps=0.0), dict(eps=NAN),
               dict(th=1e-301), dict(th=5e-324), dict(eps=INF), dict(dt=3), dict(dt=-1), dict(lq=511), dict(lq=516), dict(lk=128), dict(lqo=500)):
        assert fwd(**kw) == S, kw
    for kw in (dict(q=N), dict(gq=N), dict(pos=N), dict(qo=N), dict(rstd=N)):
        assert fwd(**kw) == NU, kw
    for kw in (dict(q=Q8), dict(gq=Q8), dict(pos=O2), dict(qo=Q8), dict(rstd=Q8)):
        assert fwd(**kw) == AL, kw
    assert fwd(T=0, q=N, pos=N, qo=N, rstd=N) == OK
    for kw in (dict(T=-1), dict(d=24), dict(rot=65), dict(th=-1.0), dict(dt=9), dict(ldy=504), dict(ldq=513)):
        assert bwd(**kw) == S, kw
    for kw in (dict(dy=N), dict(dq=N), dict(dg=N), dict(part=N)):
        assert bwd(**kw) == NU, kw
    for kw in (dict(dy=Q8), dict(dq=Q8), dict(dg=Q8), dict(part=Q8)):
        assert bwd(**kw) == AL, kw


def _clip(L, ins, outs, sizes, types, norm=P, ws=P, n_ws=1 << 40, max_norm=1.0):
    n = len(ins)
    arr = lambda xs: (ctypes.c_void_p * n)(*xs)  # noqa: E731
    return L.tp_grad_clip(arr(ins), arr(outs), (ctypes.c_longlong * n)(*sizes), (ctypes.c_int * n)(*types), n,
                          max_norm, norm, ws, n_ws, N)


def test_clip_refusals(L):
    a, b = 0x10000, 0x20000
    for kw in (dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=NAN)):
        assert _clip(L, [a], [a], [8], [0], **kw) == S
    assert _clip(L, [a], [b], [-1], [0]) == S
    assert _clip(L, [a], [b], [(1 << 40) + 1], [0]) == S
    assert _clip(L, [a], [b], [8], [3]) == S
    many = [1 << 40] * 9  # more values than the kernels count pieces of
    assert L.tp_grad_norm((ctypes.c_void_p * 9)(*[a] * 9), (ctypes.c_longlong * 9)(*many), (ctypes.c_int * 9)(), 9, P, P,
                          1 << 40, N) == S
    assert _clip(L, [0], [b], [8], [0]) == NU
    assert _clip(L, [a], [0], [8], [0]) == NU
    assert _clip(L, [a], [b], [8], [0], norm=N) == NU
    assert _clip(L, [a + 1], [b], [8], [0]) == AL
    assert _clip(L, [a], [b + 2], [8], [2]) == AL
    assert _clip(L, [a], [b], [8], [0], ws=N) == WS
    assert _clip(L, [a], [b], [8], [0], n_ws=L.tp_grad_workspace_bytes(1) - 1) == WS
    # shared memory: the same output twice, outputs that overlap, an output over
    # another tensor's gradient or over part of its own
    assert _clip(L, [a, a], [a, a], [8, 8], [0, 0]) == S
    assert _clip(L, [a, a + 64], [b, b + 14], [8, 8], [0, 0]) == S
    assert _clip(L, [a, b], [b, b + 64], [8, 8], [0, 0]) == S
    assert _clip(L, [a, b], [b + 64, a + 14], [8, 8], [0, 0]) == S
    assert _clip(L, [a], [a + 8], [8], [0]) == S
    assert L.tp_grad_norm(N, N, N, 1, P, P, 1 << 40, N) == NU
    assert L.tp_grad_norm(N, N, N, -1, P, P, 1 << 40, N) == S
    assert L.tp_grad_norm(N, N, N, 0, N, P, 1 << 40, N) == NU
    assert L.tp_grad_workspace_bytes(-1) == 0 and L.tp_grad_workspace_bytes((1 << 20) + 1) == 0


@pytest.mark.parametrize("nb,T", [(1, 1), (8, 8192), (37, 8191), (1, 1 << 20), (5000, 100)])
def test_scratch_sizes(L, nb, T):
    f = L.tp_attn_packed_forward_workspace_bytes(nb, T, 8, 2, 128)
    b = L.tp_attn_packed_backward_workspace_bytes(nb, T, 8, 2, 128)
    assert f >= 16 * (T // 128 + nb) + 4 * (T // 128 + 2) + 16
    assert b >= f + 4 * T * 8
    assert L.tp_attn_packed_forward_workspace_bytes(nb, T, 8, 3, 128) == 0
    assert L.tp_attn_packed_backward_workspace_bytes(nb, T, 8, 2, 100) == 0
    assert 0 < L.tp_qk_norm_rope_backward_workspace_floats(T, 8, 2, 128) <= 608 * 2 * 128
    assert L.tp_qk_norm_rope_backward_workspace_floats(T, 8, 2, 100) == 0


def test_parts_scratch_is_bounded(L):
    # groups dealt to parts: their fp32 sums stay near 100 MB whatever the tokens are
    plain = lambda nb, T, nh: 16 * (T // 128 + nb) + 4 * (T // 128 + 2) + 4 * T * nh + 2048  # noqa: E731
    for nb, T, nh, nkv in ((1, 128, 16, 1), (1, 8192, 16, 1), (8, 8192, 32, 8), (1, 1 << 20, 64, 1), (3, 20000, 24, 3)):
        need = L.tp_attn_packed_backward_workspace_bytes(nb, T, nh, nkv, 160)
        assert plain(nb, T, nh) - 2048 <= need <= plain(nb, T, nh) + 160 * (1 << 20), (nb, T, nh, nkv)
    # enough items without parts: nothing but the plan and delta
    assert L.tp_attn_packed_backward_workspace_bytes(1, 1 << 20, 64, 1, 160) <= plain(1, 1 << 20, 64)
    assert L.tp_attn_packed_backward_workspace_bytes(8, 8192, 16, 16, 160) <= plain(8, 8192, 16)


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        binding.tp_attn_packed_forward(x, x, x, cu)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        binding.tp_qk_norm_rope_forward(x, x, x[0, 0], x[0, 0], cu)
    with pytest.raises(ValueError, match="must be bfloat16"):
        binding.tp_qk_norm_rope_forward(x.double(), x, x[0, 0], x[0, 0], cu)
    for rot in (-16, 80, (1 << 32) + 16):  # the last is 16 in 32 bits
        with pytest.raises(ValueError, match="rot must be from 0 to d = 64"):
            binding._rotated(rot, 64)
    assert [binding._rotated(r, 64) for r in (None, 0, 48, 64)] == [64, 0, 48, 64]
    huge = torch.empty(1, dtype=torch.int32).expand((1 << 32) + 2)  # 1 sequence in 32 bits
    with pytest.raises(ValueError, match="nb"):
        binding._sequences(huge)
    with pytest.raises(ValueError, match="grads\\[0\\] is on cpu"):
        binding.tp_grad_norm([x])
