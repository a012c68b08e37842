"""A layer's attention with grouped heads on a packed batch, forward, backward and
clipped: projection, norms and rotation, attention, output projection, as a
training step runs them together (GB300)."""

import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rel(a, b):
    b = b.double()
    return float((a.double().cpu() - b.cpu()).abs().max() / b.abs().max())


@pytest.mark.parametrize("nh,nkv,d,captured", [(8, 2, 64, False), (4, 4, 128, True)])
def test_training_step(nh, nkv, d, captured):
    lens = [40, 0, 129, 1, 86]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    T, W, h = cu[-1], (nh + 2 * nkv) * d, nh * d
    g = torch.Generator().manual_seed(12)
    x = torch.randn(T, h, generator=g).to(BF)
    w = (torch.randn(h, W, generator=g) / math.sqrt(h)).to(BF)
    gq, gk = (1 + 0.1 * torch.randn(d, generator=g)).to(BF), (1 + 0.1 * torch.randn(d, generator=g)).to(BF)
    dO = torch.randn(T, nh, d, generator=g).to(BF)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])

    gpu = dict(x=x.cuda(), w=w.cuda(), gq=gq.cuda(), gk=gk.cuda(), dO=dO.cuda(), pos=pos.cuda(),
               cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), b=torch.zeros(W, dtype=BF, device="cuda"))

    def step():
        # the framework's projection has 3 h columns; of another width it is torch's
        rows = binding.tp_attn_qkv(gpu["x"], gpu["w"], gpu["b"]) if nh == nkv else torch.mm(gpu["x"], gpu["w"])
        rows = rows.view(T, nh + 2 * nkv, d)
        Q, K, V = rows[:, :nh], rows[:, nh:nh + nkv], rows[:, nh + nkv:]
        Qn, Kn, rstd = binding.tp_qk_norm_rope_forward(Q, K, gpu["gq"], gpu["gk"], gpu["pos"])
        O, lse = binding.tp_attn_packed_forward(Qn, Kn, V, gpu["cu"])
        drows = torch.empty_like(rows)
        dQn, dKn, _ = binding.tp_attn_packed_backward(Qn, Kn, V, O, lse, gpu["dO"], gpu["cu"], dV=drows[:, nh + nkv:])
        _, _, dgq, dgk = binding.tp_qk_norm_rope_backward(dQn, dKn, Q, K, gpu["gq"], gpu["gk"], gpu["pos"], rstd,
                                                          dQ=drows[:, :nh], dK=drows[:, nh:nh + nkv])
        dW = binding.tp_mlp_dA_ws(gpu["x"], drows.view(T, W), 1)
        db = binding.tp_mlp_bias_grad(drows.view(T, W))
        grads = [dW, db, dgq, dgk]
        raw = [t.clone() for t in grads]
        norm, _ = binding.tp_grad_clip(grads, 1.0)
        return O, drows, raw, norm, grads

    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            O, drows, raw, norm, grads = step()
        graph.replay()
        graph.replay()
    else:
        O, drows, raw, norm, grads = step()
    torch.cuda.synchronize()
    assert binding.device_status() == 0

    # 64 bits from the same inputs, nothing rounded in between
    rows = (x.double() @ w.double()).view(T, nh + 2 * nkv, d)
    q, k, v = rows[:, :nh], rows[:, nh:nh + nkv], rows[:, nh + nkv:]
    qn, rq, _ = ref.qk_forward(q, gq, pos, d, 1e4, 1e-5)
    kn, rk, _ = ref.qk_forward(k, gk, pos, d, 1e4, 1e-5)
    o, lse, _ = ref.attention(qn, kn, v, cu, d ** -0.5)
    (dqn, dkn, dv), _ = ref.attention_backward(qn, kn, v, o, lse, dO, cu, d ** -0.5)
    dq, dgq, _, _ = ref.qk_backward(dqn, q, gq, pos, rq, d, 1e4)
    dk, dgk, _, _ = ref.qk_backward(dkn, k, gk, pos, rk, d, 1e4)
    want = torch.cat([dq, dk, dv], 1)
    # four roundings to bf16 one behind another, as the framework's blocks are held to
    assert _rel(O, o) <= 2e-2 and _rel(drows, want) <= 3e-2
    for a, b in zip(raw, (x.double().t() @ want.reshape(T, W), want.reshape(T, W).sum(0), dgq, dgk)):
        assert _rel(a, b) <= 3e-2
    total = math.sqrt(sum(float((t.double() ** 2).sum()) for t in raw))
    assert total > 1.0 and abs(float(norm) - total) <= 2.0 ** -17 * total
    for a, b in zip(grads, raw):
        assert ((a.double() - b.double() / total).abs() <= (2.0 ** -8 + 2.0 ** -16) * b.double().abs() / total
                + 1e-30 + 2e-6 * b.double().abs()).all()
