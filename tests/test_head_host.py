"""Refusals and scratch sizes of the final norm and the output head, on a host
without a GPU: every bad argument is answered before CUDA is touched."""

import ctypes

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding, build

P = ctypes.c_void_p(0x10000)
Q = ctypes.c_void_p(0x10008)  # 8-byte aligned only
N = None
S, NU, AL, WS, OK = (binding.TPMLP_ERR_SHAPE, binding.TPMLP_ERR_NULL, binding.TPMLP_ERR_ALIGN,
                     binding.TPMLP_ERR_WORKSPACE, binding.TPMLP_OK)


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def test_norm_refusals(L):
    fwd = lambda x=P, g=P, T=4, h=24, dt=0, eps=1e-5, y=P, m=P: L.tp_ln_forward(  # noqa: E731
        x, g, P, T, h, dt, eps, y, m, P, N)
    for kw in (dict(T=-1), dict(h=0), dict(h=-8), dict(dt=-1), dict(dt=3), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=float("nan"))):
        assert fwd(**kw) == S, kw
    for kw in (dict(x=N), dict(g=N), dict(y=N), dict(m=N)):
        assert fwd(**kw) == NU, kw
    for kw in (dict(x=Q), dict(g=Q), dict(y=Q)):
        assert fwd(**kw) == AL, kw
    assert fwd(T=0, x=N, y=N, m=N) == OK
    bwd = lambda dy=P, T=4, h=24, dt=0, dx=P, dg=P, part=P: L.tp_ln_backward(  # noqa: E731
        dy, P, P, P, P, T, h, dt, dx, dg, P, part, N)
    for kw in (dict(T=-1), dict(h=0), dict(dt=7)):
        assert bwd(**kw) == S, kw
    for kw in (dict(dy=N), dict(dx=N), dict(dg=N), dict(part=N)):
        assert bwd(**kw) == NU, kw
    for kw in (dict(dy=Q), dict(dx=Q), dict(dg=Q), dict(part=Q)):
        assert bwd(**kw) == AL, kw
    assert L.tp_ln_backward_workspace_floats(-1, 8, 0) == 0
    assert L.tp_ln_backward_workspace_floats(4, 8, 3) == 0
    for T, h in ((1, 1), (8192, 1024), (2048, 20480), (3, 50001)):
        assert L.tp_ln_backward_workspace_floats(T, h, 0) >= 2 * h


def test_head_refusals(L):
    big = 1 << 40
    fwd = lambda X=P, W=P, y=P, T=4, h=24, V=100, lo=P, ws=P, n=big: L.tp_head_loss_forward(  # noqa: E731
        X, W, y, T, h, V, lo, P, ws, n, N)
    for kw in (dict(T=-1), dict(h=0), dict(h=12), dict(V=0), dict(V=-3), dict(V=(1 << 30) + 1)):
        assert fwd(**kw) == S, kw
    for kw in (dict(X=N), dict(W=N), dict(y=N), dict(lo=N)):
        assert fwd(**kw) == NU, kw
    for kw in (dict(X=Q), dict(W=Q), dict(ws=Q)):
        assert fwd(**kw) == AL, kw
    need = L.tp_head_loss_forward_workspace_bytes(4, 24, 100)
    assert need > 0
    assert fwd(ws=N) == WS and fwd(n=need - 1) == WS
    assert fwd(T=0, X=N, y=N, lo=N, ws=N, n=0) == OK
    bwd = lambda dl=P, X=P, T=4, h=24, V=100, dX=P, dW=P, ws=P, n=big: L.tp_head_loss_backward(  # noqa: E731
        dl, X, P, P, P, T, h, V, dX, dW, ws, n, N)
    for kw in (dict(T=-1), dict(h=20), dict(V=0)):
        assert bwd(**kw) == S, kw
    for kw in (dict(dl=N), dict(X=N), dict(dX=N), dict(dW=N)):
        assert bwd(**kw) == NU, kw
    for kw in (dict(X=Q), dict(dX=Q), dict(dW=Q), dict(ws=Q)):
        assert bwd(**kw) == AL, kw
    least = L.tp_head_loss_backward_min_workspace_bytes(4, 24, 100)
    assert bwd(ws=N) == WS and bwd(n=least - 1) == WS


@pytest.mark.parametrize("T,h,V", [(1, 8, 1), (1, 1024, 50257), (7, 1024, 50257), (8192, 1024, 50257),
                                   (2048, 20480, 51200), (100000, 64, 131072), (333, 4096, 32003)])
def test_head_scratch_sizes(L, T, h, V):
    full = L.tp_head_loss_backward_workspace_bytes(T, h, V)
    least = L.tp_head_loss_backward_min_workspace_bytes(T, h, V)
    assert 0 < least <= full
    # one piece of at least 256 columns (or the vocabulary)
    assert least >= 2 * T * min(256, V)
    # pieces of at most 512 MiB (and the rounding to 256 columns), and dX's
    # fp32 planes, never the logits of a large batch
    assert full <= (512 << 20) + 2 * T * 256 + 608 * 4 * T * max(h, 256) + 16 * T + 4096
    # row statistics of each half tile, or of each CTA at few tokens
    assert 0 < L.tp_head_loss_forward_workspace_bytes(T, h, V) <= 18 * T * max(-(-V // 256), 304)


def test_no_work_for_bad_sizes(L):
    for f in (L.tp_head_loss_forward_workspace_bytes, L.tp_head_loss_backward_workspace_bytes,
              L.tp_head_loss_backward_min_workspace_bytes):
        assert f(4, 12, 100) == 0 and f(-1, 24, 100) == 0 and f(4, 24, 0) == 0


def test_binding_refusals():
    x = torch.zeros(4, 24, dtype=torch.float64)
    with pytest.raises(ValueError, match="must be bfloat16"):
        binding.tp_ln_forward(x, x[0], x[0])
    b = torch.zeros(4, 24, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        binding.tp_ln_forward(b, b[0], b[0], y=b, mean=b[0], rstd=b[0])
