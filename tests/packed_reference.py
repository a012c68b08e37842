"""Plain 64-bit forms (CPU) of packed grouped attention, the norms and rotation
of queries and keys, and gradient clipping, with the sums that bound the
kernels' rounding errors."""

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step


def _visible(n):
    return torch.ones(n, n, dtype=torch.bool).tril()


def attention(Q, K, V, cu, scale):
    """O, lse (log2) and A = sum_k P |V|; rows in no sequence are NaN."""
    Q, K, V = Q.double(), K.double(), V.double()
    T, nh, d = Q.shape
    g = nh // K.shape[1]
    O = torch.full_like(Q, math.nan)
    A = torch.zeros_like(Q)
    lse = torch.full((nh, T), math.nan, dtype=torch.float64)
    for a, b in zip(cu, cu[1:]):
        for j in range(nh if b > a else 0):
            z = Q[a:b, j] @ K[a:b, j // g].t() * scale
            z = torch.where(_visible(b - a), z, torch.tensor(-math.inf, dtype=torch.float64))
            s = torch.logsumexp(z, 1)
            p = torch.exp(z - s[:, None])
            O[a:b, j] = p @ V[a:b, j // g]
            A[a:b, j] = p @ V[a:b, j // g].abs()
            lse[j, a:b] = s / math.log(2.0)
    return O, lse, A


def attention_backward(Q, K, V, O, lse, dO, cu, scale, two=False):
    """dQ, dK, dV from the saved O and lse, and a bound of the errors of each: its
    operands P and dS are rounded to bf16 (half a step each), dP, delta and the
    exponents to fp32 (sums of d <= 160 terms), the result to bf16.  two: dS is held
    in two bf16 parts, of which the second's rounding is 2^-8 of 2^-8 off."""
    Q, K, V, O, dO, lse = (x.double() for x in (Q, K, V, O, dO, lse))
    T, nh, d = Q.shape
    g = nh // K.shape[1]
    out = [torch.zeros_like(x) for x in (Q, K, V)]
    half, wide = 2.0 ** -8 * (1 + 2.0 ** -6) + 2.0 ** -12, 2.0 ** -15
    tol = [torch.zeros_like(x) for x in (Q, K, V)]
    for a, b in zip(cu, cu[1:]):
        for j in range(nh if b > a else 0):
            q, k, v, do = Q[a:b, j], K[a:b, j // g], V[a:b, j // g], dO[a:b, j]
            p = torch.exp2(q @ k.t() * scale / math.log(2.0) - lse[j, a:b, None]) * _visible(b - a)
            delta = (do * O[a:b, j]).sum(1, keepdim=True)
            ds = p * (do @ v.t() - delta)
            # |dS| as rounded, and the fp32 error of dP - delta
            e = (2.0 ** -16 + 2.0 ** -12 if two else half) * ds.abs() + wide * p * (do.abs() @ v.abs().t() + (do * O[a:b, j]).abs().sum(1, keepdim=True))
            out[0][a:b, j] = ds @ k * scale
            tol[0][a:b, j] = e @ k.abs() * scale
            out[1][a:b, j // g] += ds.t() @ q * scale
            tol[1][a:b, j // g] += e.t() @ q.abs() * scale
            out[2][a:b, j // g] += p.t() @ do
            tol[2][a:b, j // g] += half * (p.t() @ do.abs())
    for x, t in zip(out, tol):
        t += 2.0 ** -8 * (x.abs() + t)
    return out, tol


def _turn(x, positions, rot, theta, sign):
    h = rot // 2
    if h == 0:
        return x
    a = positions.double()[:, None] * theta ** (-2.0 * torch.arange(h, dtype=torch.float64) / rot) * sign
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    u, w = x[..., :h], x[..., h:rot]
    return torch.cat([u * c - w * s, w * c + u * s, x[..., rot:]], -1)


def qk_forward(x, gamma, positions, rot, theta, eps):
    """y, rstd and the size |u_i| + |u_{i + rot/2}| that an element's rotation mixes."""
    x, gamma = x.double(), gamma.double()
    rstd = 1.0 / torch.sqrt((x * x).mean(-1) + eps)
    u = x * rstd[..., None] * gamma
    return _turn(u, positions, rot, theta, 1.0), rstd, _mixed(u, rot)


def _mixed(u, rot):
    h = rot // 2
    m = u.abs()
    both = m[..., :h] + m[..., h:rot]
    return torch.cat([both, both, m[..., rot:]], -1)


def qk_backward(dy, x, gamma, positions, rstd, rot, theta):
    """dx, dgamma and sizes of their terms."""
    dy, x, gamma, r = dy.double(), x.double(), gamma.double(), rstd.double()[..., None]
    g = _turn(dy, positions, rot, theta, -1.0)
    size = _mixed(dy, rot)
    xhat = x * r
    gg = g * gamma
    m = (gg * xhat).mean(-1, keepdim=True)
    dx = r * (gg - xhat * m)
    dx_size = r * (size * gamma.abs() + xhat.abs() * (size * gamma.abs() * xhat.abs()).mean(-1, keepdim=True))
    return dx, (g * xhat).sum((0, 1)), dx_size, (size * xhat.abs()).sum((0, 1))
