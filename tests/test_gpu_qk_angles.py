"""The angles of the rotation of queries and keys, against angles reduced in 60 digits
(GB300)."""

import decimal
import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding

pytestmark = pytest.mark.gpu
D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")
FAR = (2**31 - 1, -2**31, 2**30 + 12345, 1234567891, -987654321, 16777217)


def _turns(positions, rot, theta):
    """cos and sin [T, rot / 2] in 64 bits."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        freq = [(D(-2 * i) / rot * D(theta).ln()).exp() / (2 * PI) for i in range(rot // 2)]
        out = torch.empty(2, len(positions), rot // 2, dtype=torch.float64)
        for t, p in enumerate(positions):
            for i, f in enumerate(freq):
                turn = p * f
                quarter = int((4 * turn).to_integral_value(decimal.ROUND_HALF_EVEN))
                rest = float(2 * PI * (turn - D(quarter) / 4))  # at most an eighth of a turn
                c, s = math.cos(rest), math.sin(rest)
                c, s = ((c, s), (-s, c), (-c, -s), (s, -c))[quarter % 4]
                out[0, t, i], out[1, t, i] = c, s
    return out


def _rotated(x, positions, rot, theta):
    """Q and K of the same values [T, 1, d], gamma 1, and what rstd x makes in 64 bits."""
    T, d = len(positions), x.shape[2]
    one = torch.ones(d, dtype=x.dtype, device="cuda")
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    Q, K, rstd = binding.tp_qk_norm_rope_forward(x.cuda(), x.cuda(), one, one, pos, rot=rot, theta=theta, eps=1e-20)
    u = x.double() * rstd.double().cpu()[:, :1, None]
    a, b = u[:, 0, :rot // 2], u[:, 0, rot // 2:rot]
    c, s = _turns(positions, rot, theta)
    assert torch.equal(Q, K) and torch.equal(Q[..., rot:].double().cpu(), u.to(x.dtype)[..., rot:].double())
    return Q.double().cpu()[:, 0, :rot], torch.cat([a * c - b * s, b * c + a * s], 1), torch.cat([a.abs() + b.abs()] * 2, 1)


# angle: rounded to fp32 (2^-24 of an eighth of a turn, pi / 4) and 2^-33 turns; sine and
# cosine two last bits of at most 1; two roundings of products and sums
ABSOLUTE = 2.0 ** -24 * math.pi / 4 + 2 * math.pi * 2.0 ** -33 + 2.0 ** -23 + 2 * 2.0 ** -24


@pytest.mark.parametrize("first", [0.0, 1.0])
@pytest.mark.parametrize("d,rot,theta", [(96, 96, 5e5), (128, 128, 1e4), (256, 256, 1e6), (64, 32, 1e4), (32, 32, 1.5)])
def test_far_positions(d, rot, theta, first):
    g = torch.Generator().manual_seed(d)
    x = (torch.randint(0, 2, (len(FAR), 1, d), generator=g) * 2 - 1).float()
    x[..., :rot // 2] *= first
    got, want, size = _rotated(x, FAR, rot, theta)
    assert ((got - want).abs() <= ABSOLUTE * size).all()


@pytest.mark.parametrize("dt,half", [(torch.float32, 2.0 ** -24), (torch.float16, 2.0 ** -11), (torch.bfloat16, 2.0 ** -8)])
@pytest.mark.parametrize("d,rot,theta", [(256, 256, 1e6), (128, 64, 1e4)])
def test_small_angles_keep_their_digits(dt, half, d, rot, theta):
    # a value that is the sine of its angle alone, angles from 1e-6 on
    positions = (0, 1, -1, 2, 3, 7, 100, -1000, 65537)
    x = torch.ones(len(positions), 1, d, dtype=dt)
    x[..., :rot // 2] = 0.0
    got, want, size = _rotated(x, positions, rot, theta)
    # the angle's rounding and the result's product, 2^-24 each, the sine's two last bits
    # (2^-22 of it), and the frequency's 2^-64 of a turn (with the reduction's, twice);
    # then the result's own, half a step of a normal value or of the smallest one
    slack = 2 * 2.0 ** -24 + 2.0 ** -22
    tiny = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[dt]
    bound = (half * (1 + 2.0 ** -10) + slack) * want.abs() + tiny
    bound += size * (4 * math.pi * 2.0 ** -64 * torch.tensor(positions).abs().double())[:, None]
    assert ((got - want).abs() <= bound).all()
