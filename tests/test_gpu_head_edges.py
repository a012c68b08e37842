"""The output head where it can go wrong beside plain batches: tokens that the
model is sure of."""

import numpy as np
import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import head_reference as ref

pytestmark = pytest.mark.gpu


def lean_on(T, h, V, seed, logit):
    """Tokens whose targets have logits of about `logit`, one in ten ignored."""
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, h, generator=g) * 0.64 / h ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g)
    Wt = W[y].float()
    X = torch.randn(T, h, generator=g) + logit * Wt / (Wt * Wt).sum(-1, keepdim=True)
    y = torch.where(torch.rand(T, generator=g) < 0.1, torch.full_like(y, -1), y)
    return dict(X=X.to(torch.bfloat16), W=W, y=y, dloss=(0.5 + torch.rand(T, generator=g)) / T)


@pytest.mark.parametrize("T,h,V", [(40, 20480, 1500), (64, 4096, 1501), (300, 1024, 3001), (1000, 2048, 1003)])
def test_gradients_of_sure_tokens(T, h, V):
    """Targets with logits of 16, so that 1 - p is about 2e-4: the target's dz
    = p - 1 has an error of its own, far below the 4e-4 by which a tensor-core
    accumulator of 20480 products is off.

    Its logit is a sum over 128 threads or more in fp32.  A thread adds at
    most 90 terms to partial sums below 1/4 (1/2 with 1024 products, 9 terms
    each), each rounding at most 2^-27 (2^-26): the roundings of all
    threads, added in squares, are below 7e-7, six times that is 4e-6; the
    threads' sums meet exactly to 2^-48.  z - lse is exact and its expm1 off
    by 2^-22: 5e-6 in all.  The other classes' p carry the accumulator's error,
    relative to p.  Bounds for every value of dX and dW as in head_reference."""
    c = lean_on(T, h, V, h + T, 16.0)
    d = {k: v.cuda() for k, v in c.items()}
    _, lse = binding.tp_head_loss_forward(d["X"], d["W"], d["y"])
    dX, dW = binding.tp_head_loss_backward(d["dloss"], d["X"], d["W"], d["y"], lse)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    X, W, dl, s, y = (ref.f64(v) for v in (c["X"], c["W"], c["dloss"], lse, c["y"]))
    y = y.astype(int)
    r = np.nonzero(y >= 0)[0]
    z = X @ W.T
    p = np.exp(z - s[:, None])
    p[y < 0] = 0.0
    ez = ref.logit_bound(X, W) + 2.0 ** -21 * (2 + np.abs(z) + np.abs(s)[:, None])
    e = p * ez * (1 + 2 * ez)
    p[r, y[r]] = np.expm1(z[r, y[r]] - s[r])
    e[r, y[r]] = 5e-6
    assert 5e-5 < float(np.median(-p[r, y[r]])) < 1e-3
    dz, e, u = p * dl[:, None], e * dl[:, None], ref.U[torch.bfloat16]
    e = e + 2.0 ** -22 * np.abs(dz)
    e = e + u * (np.abs(dz) + e)
    a = np.abs(dz) + e
    for got, ez_out, sums, want, n, name in ((dX, e @ np.abs(W), a @ np.abs(W), dz @ W, V, "dX"),
                                             (dW, e.T @ np.abs(X), a.T @ np.abs(X), dz.T @ X, T, "dW")):
        bound = (1 + u) * (ez_out + (n / 16 + 80) * 2.0 ** -23 * sums) + u * np.abs(want) + 1e-37
        ref.within(got, want, bound, name)


def test_two_calls_at_once_from_dirty_workspaces():
    """Rows wide enough for grids whose CTAs take one another's tiles over
    (12288 values and more), two calls side by side on two streams with
    workspaces full of NaN: the largest weight and every other intermediate
    come from the call itself, whichever of its CTAs run first."""
    T, h, V = 300, 12296, 6001
    cs = [{k: v.cuda() for k, v in lean_on(T, h, V, s, 4.0).items()} for s in (1, 2)]
    lses = [binding.tp_head_loss_forward(c["X"], c["W"], c["y"])[1] for c in cs]
    want = [binding.tp_head_loss_backward(c["dloss"], c["X"], c["W"], c["y"], s) for c, s in zip(cs, lses)]
    n = binding.head_loss_backward_workspace_bytes(T, h, V)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        ws = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in cs]
        torch.cuda.synchronize()
        got = [binding.tp_head_loss_backward(c["dloss"], c["X"], c["W"], c["y"], s, workspace=w, stream=st)
               for c, s, w, st in zip(cs, lses, ws, streams)]
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T", [17, 257, 2049, 9000])
def test_the_largest_weight_may_be_any_token_s(T):
    """One weight far above the others, at the first, last or a middle token,
    and a larger one at a token that does not count: the same gradients as
    with all weights and results scaled by a power of two, bit for bit."""
    h, V = 64, 300
    c = {k: v.cuda() for k, v in lean_on(T, h, V, T, 4.0).items()}
    _, lse = binding.tp_head_loss_forward(c["X"], c["W"], c["y"])
    for at in (0, T // 2, T - 1):
        y = c["y"].clone()
        y[at] = 7
        y[(at + 5) % T] = -1
        dl = c["dloss"].clone()
        dl[at], dl[(at + 5) % T] = 2.0, 1e9
        want = binding.tp_head_loss_backward(dl, c["X"], c["W"], y, lse)
        got = binding.tp_head_loss_backward(dl * 1024.0, c["X"], c["W"], y, lse)
        for a, b in zip(got, want):
            assert torch.equal(a.float(), 1024.0 * b.float()) and bool(a.float().abs().max() > 0)


@pytest.mark.parametrize("T,h,V,classes", [(40, 20480, 1500, (0, 700)), (90, 20480, 1500, (0, 300, 900)),
                                           (700, 8192, 1501, (0, 520)), (6200, 4096, 600, (0, 300)),
                                           (12300, 4096, 600, (0,)), (12200, 2048, 1027, (5,))])
def test_rows_torn_between_classes(T, h, V, classes):
    """Rows with equal logits of about 20 at a few classes far apart, none of
    them the target (every third row counts, every third counts for one of
    them); up to 32 rows a CTA.  All of these logits are taken again in fp32.

    A lane adds at most 9 h / 256 rounded terms to partial sums below 1 (20 of
    32 lanes and the noise): at most 720 roundings of 2^-25 in 32 lanes, in
    squares 2.6e-6 for h = 20480, six times that is 1.6e-5 or 2^-20.3 of a
    logit of 20.  lse's own roundings and the 2^x of the sum: 2^-21 of it.  The
    others' logits shift by less than 2^-18 of their size, 1, times their share,
    below 2^-8: together below 2^-19 relative."""
    g = torch.Generator().manual_seed(T + h)
    W = (torch.randn(V, h, generator=g) * 0.64 / h ** 0.5).to(torch.bfloat16)
    base = torch.randint(0, V - max(classes) - 1, (T,), generator=g)
    # W's rows are nearly orthogonal: their pseudo-inverse gives each its logit
    cols = base[:, None] + torch.tensor(classes)
    S = W[cols].float()  # [T, classes, h]
    gram = S @ S.transpose(1, 2)
    X = torch.randn(T, h, generator=g)
    X = X + (torch.linalg.solve(gram, 20.0 - (S @ X[:, :, None])).transpose(1, 2) @ S)[:, 0]
    kind = torch.arange(T) % 3
    y = torch.where(kind == 0, torch.full_like(base, -1), torch.where(kind == 1, base, base + max(classes) + 1))
    d = [t.cuda() for t in (X.to(torch.bfloat16), W, y)]
    loss, lse = binding.tp_head_loss_forward(*d)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    z = d[0].double() @ d[1].double().T
    want = torch.logsumexp(z, 1)
    # the share of the classes: nothing else matters
    assert float(torch.exp(z.gather(1, cols.cuda()) - want[:, None]).sum(1).min()) > 1 - 2.0 ** -8
    off = float(((lse.double() - want) / want).abs().max())
    assert off <= 2.0 ** -19, off
    rest = z.clone()
    counted = d[2] >= 0
    at = d[2].clamp(min=0)[:, None]
    zt = z.gather(1, at)[:, 0]
    rest.scatter_(1, at, torch.where(counted, torch.full_like(zt, -torch.inf), zt)[:, None])
    want_loss = torch.where(counted, torch.nn.functional.softplus(torch.logsumexp(rest, 1) - zt), torch.zeros_like(zt))
    off = float((loss.double() - want_loss).abs().max() / want.max())
    assert off <= 2.0 ** -19, off


@pytest.mark.parametrize("T,h,V", [(9, 264, 999), (9, 2056, 999), (150, 264, 999), (300, 64, 5003)])
def test_a_bad_token_stays_by_itself(T, h, V):
    """A counted token's row of NaN, its weight of infinity: its own loss, lse and
    dX are NaN, the other tokens' bit for bit as without it.  (dW's rows sum all
    tokens: NaN.)"""
    c = {k: v.cuda() for k, v in lean_on(T, h, V, T, 4.0).items()}
    c["y"][3] = 5
    loss0, lse0 = binding.tp_head_loss_forward(c["X"], c["W"], c["y"])
    X = c["X"].clone()
    X[3] = float("nan")
    loss, lse = binding.tp_head_loss_forward(X, c["W"], c["y"])
    ok = torch.arange(T, device="cuda") != 3
    assert torch.equal(loss[ok], loss0[ok]) and torch.equal(lse[ok], lse0[ok])
    assert bool(torch.isnan(loss[3])) and bool(torch.isnan(lse[3]))
    dX0, _ = binding.tp_head_loss_backward(c["dloss"], c["X"], c["W"], c["y"], lse0)
    dX, dW = binding.tp_head_loss_backward(c["dloss"], X, c["W"], c["y"], lse)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    assert torch.equal(dX[ok], dX0[ok]) and bool(torch.isnan(dX[3].float()).all())
    assert bool(torch.isnan(dW.float()).all())
