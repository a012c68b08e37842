"""Plain float64 forms of the final LayerNorm and of the output head's loss,
and the error bounds that the tests hold the kernels to.

Bounds.  A rounding to type t is off by at most u_t = eps_t / 2 relative to
the value.  An fp32 sum of n terms, added along chains of at most k additions,
is off by at most k 2^-24 times the sum of the terms' sizes (first order).  A
tensor-core accumulator may truncate: 2^-23 for each of its steps of 16 terms.
"""

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24


def f64(x):
    return x.detach().to("cpu", torch.float64).numpy()


# --------------------------------------------------------------- LayerNorm

def ln_forward(x, gamma, beta, eps):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    return c * rstd[:, None] * gamma + beta, mean, rstd


def ln_backward(dy, x, gamma, mean, rstd):
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(1)[:, None] - xhat * (g * xhat).mean(1)[:, None])
    return dx, (dy * xhat).sum(0), dy.sum(0)


def ln_forward_bounds(x, gamma, beta, eps, dtype):
    """Bounds of |y|, |mean|, |rstd| errors: sums of h terms in chains of at
    most h / 8 + 16 additions (eight threads a row at the least), a handful
    of roundings each for xhat, the scale and the shift."""
    y, mean, rstd = ln_forward(x, gamma, beta, eps)
    k = (x.shape[1] / 8 + 16) * F32
    e_mean = k * np.abs(x).mean(1)
    # var's relative error: its own sum, and x - mean off by e_mean
    e_rstd = rstd * (k + 4 * F32 + (e_mean * rstd) ** 2)
    xhat = np.abs(x - mean[:, None]) * rstd[:, None]
    e = (e_mean * rstd)[:, None] * np.abs(gamma) + xhat * np.abs(gamma) * ((e_rstd / rstd)[:, None] + 4 * F32)
    e = e + F32 * (np.abs(x).max(1) * rstd)[:, None] * np.abs(gamma) + 2 * F32 * np.abs(beta)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0  # half a step of the subnormals
    return (1 + U[dtype]) * e + U[dtype] * np.abs(y) + tiny, e_mean, e_rstd


def ln_backward_bounds(dy, x, gamma, mean, rstd, dtype):
    """Bounds for dx (mean and rstd as given), dgamma, dbeta."""
    T, h = x.shape
    dx, _, _ = ln_backward(dy, x, gamma, mean, rstd)
    k = (h / 8 + 20) * F32
    xhat = np.abs(x - mean[:, None]) * rstd[:, None]
    g = np.abs(dy * gamma)
    e = rstd[:, None] * (4 * F32 * g + k * g.mean(1)[:, None] + (k + 4 * F32) * xhat * (g * xhat).mean(1)[:, None])
    e = e + 4 * F32 * np.abs(dx)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    kt = (T + 16) * F32
    return ((1 + U[dtype]) * e + U[dtype] * np.abs(dx) + tiny, kt * (np.abs(dy) * xhat).sum(0) + 1e-30,
            kt * np.abs(dy).sum(0) + 1e-30)


# -------------------------------------------------------------- loss of logits

def loss_forward(X, W, y):
    """loss as log(1 + sum_{v != y} exp(z_v - z_y)): lse - z_y would lose a
    small loss to cancellation in float64 too (2^-53 of a logit of 30 is
    3e-15, more than the loss of a token with logit 40 itself)."""
    z = X @ W.T
    m = z.max(1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(1))
    rows, col = np.arange(len(y)), np.maximum(y, 0)
    zy = z[rows, col]
    rest = z.copy()
    rest[rows, col] = -np.inf
    mr = np.where(np.isfinite(rest.max(1)), rest.max(1), 0.0)
    with np.errstate(divide="ignore"):  # one class: nothing beside the target
        d = mr + np.log(np.exp(rest - mr[:, None]).sum(1)) - zy
    return np.where(y >= 0, np.maximum(d, 0.0) + np.log1p(np.exp(-np.abs(d))), 0.0), lse, z


def loss_backward(dloss, X, W, y, lse):
    """dX, dW and the weights-relative dz (by the largest counted |dloss|)."""
    w = np.where(y >= 0, dloss, 0.0)
    p = np.exp(X @ W.T - lse[:, None])
    one = np.zeros_like(p)
    one[np.arange(len(y)), np.maximum(y, 0)] = 1.0
    dz = (p - one) * w[:, None]
    return dz @ W, dz.T @ X, dz, p * np.abs(w)[:, None]


def logit_bound(X, W):
    """Bound of a logit's error: h / 16 accumulation steps, each cut by at
    most 2^-23 of the partial sum, which |X| |W|^T bounds."""
    return (X.shape[1] / 16 + 4) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T)


def loss_forward_bounds(X, W, y):
    """lse: a softmax average of the logits' errors, at most the largest; the
    exponentials and their sum add a few 2^-21 relative (the 2^x
    approximation and the rounding of its argument, about 2^-22 |z|).  loss =
    log(1 + sum exp(z_v - z_y)): its derivative is 1 - p_y <= loss.  A loss
    below fp32's smallest normal number, 2^-126, may come out as 0."""
    loss, lse, z = loss_forward(X, W, y)
    e = logit_bound(X, W).max(1) + 2.0 ** -21 * (1 + np.abs(z).max(1))
    return (2 * e * np.minimum(1.0, loss) + 2.0 ** -21 * loss + 2.0 ** -126, e + 2.0 ** -21 * np.abs(lse))


def loss_backward_bounds(dloss, X, W, y, lse):
    """dz is rounded to bf16 once (u), p carries its exponent's error; the
    sums over V (dX) and T (dW) accumulate in steps of 16; the outputs are
    rounded once more."""
    u = U[torch.bfloat16]
    dX, dW, dz, pw = loss_backward(dloss, X, W, y, lse)
    ez = logit_bound(X, W) + 2.0 ** -21 * (2 + np.abs(X @ W.T) + np.abs(lse)[:, None])
    e = pw * ez * (1 + 2 * ez) + 2.0 ** -22 * np.abs(dz)
    e = e + u * (np.abs(dz) + e)
    a = np.abs(dz) + e
    T, V = dz.shape
    eX = e @ np.abs(W) + (V / 16 + 80) * 2.0 ** -23 * (a @ np.abs(W))
    eW = e.T @ np.abs(X) + (T / 16 + 80) * 2.0 ** -23 * (a.T @ np.abs(X))
    return (1 + u) * eX + u * np.abs(dX) + 1e-37, (1 + u) * eW + u * np.abs(dW) + 1e-37


def within(got, ref, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), (
        f"{what}: {int((over > 0).sum())} of {over.size} values beyond their bound, worst "
        f"{float(np.max(np.abs(got - ref) / bound)):.3g} times")
