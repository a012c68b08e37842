"""LayerNorm without a residual against its float64 form, through the C ABI."""

import numpy as np
import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import head_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def draw(T, h, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(T, h) * (0.5 + 2 * torch.rand(T, 1, generator=g)) + 0.3 * r(T, 1)).to(dtype)
    return dict(x=x, gamma=(1 + 0.1 * r(h)).to(dtype), beta=(0.1 * r(h)).to(dtype),
                dy=r(T, h).to(dtype))


def check(T, h, dtype, seed=None):
    c = draw(T, h, dtype, T + h if seed is None else seed)
    g = {k: v.cuda() for k, v in c.items()}
    y, mean, rstd = binding.tp_ln_forward(g["x"], g["gamma"], g["beta"], EPS)
    dx, dgamma, dbeta = binding.tp_ln_backward(g["dy"], g["x"], g["gamma"], mean, rstd)
    torch.cuda.synchronize()
    d = {k: ref.f64(v) for k, v in c.items()}
    yr, mr, rr = ref.ln_forward(d["x"], d["gamma"], d["beta"], EPS)
    by, bm, br = ref.ln_forward_bounds(d["x"], d["gamma"], d["beta"], EPS, dtype)
    ref.within(y, yr, by, "y")
    ref.within(mean, mr, bm, "mean")
    ref.within(rstd, rr, br, "rstd")
    m, r = ref.f64(mean), ref.f64(rstd)  # the backward pass takes them as given
    out = ref.ln_backward(d["dy"], d["x"], d["gamma"], m, r)
    bounds = ref.ln_backward_bounds(d["dy"], d["x"], d["gamma"], m, r, dtype)
    for got, want, b, name in zip((dx, dgamma, dbeta), out, bounds, ("dx", "dgamma", "dbeta")):
        ref.within(got, want, b, name)


# one value a row, fewer than a vector, odd widths, whole vectors, the widths
# where a row takes another number of threads or registers, very long rows;
# one row, fewer rows than SMs, ragged counts
SHAPES = [(1, 1), (5, 3), (3, 8), (1, 4096), (1, 20480), (37, 200), (130, 255), (300, 1024), (5, 1023),
          (257, 1032), (64, 2047), (9, 4100), (33, 8192), (70, 8200), (200, 9001), (5, 16392), (3, 12289), (17, 20480),
          (2, 24576), (3, 32776), (2, 50001), (1000, 64), (2051, 40)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h", SHAPES)
def test_against_float64(T, h, dtype):
    check(T, h, dtype)


# numbers of warps that are no power of two, clusters of each even size with
# whole and ragged shares, the widest rows in registers and the first beyond
WIDTHS = [(40, 2560), (12, 3333), (9, 3000), (31, 5120), (31, 6152), (11, 10240), (7, 12296), (5, 14336),
          (4, 18432), (3, 28680), (2, 40968), (2, 65536), (2, 65544)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h", WIDTHS)
def test_warps_and_clusters(T, h, dtype):
    check(T, h, dtype)


@pytest.mark.parametrize("T,h,dtype", [(8192, 1024, torch.bfloat16), (2048, 20480, torch.bfloat16),
                                       (20000, 72, torch.float16), (1031, 4100, torch.float32)])
def test_training_batches(T, h, dtype):
    check(T, h, dtype)


def test_one_value_a_row_is_exact():
    """h = 1: x is its own mean, so y is beta and dx is 0, without residue."""
    x = torch.randn(77, 1, device="cuda") * 100
    gam, bet = torch.full((1,), 1.3, device="cuda"), torch.full((1,), 0.7, device="cuda")
    y, mean, rstd = binding.tp_ln_forward(x, gam, bet, EPS)
    dx, dgamma, dbeta = binding.tp_ln_backward(torch.randn_like(x), x, gam, mean, rstd)
    assert torch.equal(y, bet.expand_as(y)) and torch.equal(mean, x[:, 0])
    assert float(dx.abs().max()) == 0.0 and float(dgamma.abs().max()) == 0.0


def test_large_offset_keeps_the_variance():
    """Rows whose mean is far larger than their spread: the variance is taken
    from x - mean, not from a difference of squares."""
    T, h = 64, 1024
    c = draw(T, h, torch.float32, 3)
    x = (c["x"] + 1000.0).cuda()
    y, mean, rstd = binding.tp_ln_forward(x, c["gamma"].cuda(), c["beta"].cuda(), EPS)
    d = ref.f64(x)
    yr, mr, rr = ref.ln_forward(d, ref.f64(c["gamma"]), ref.f64(c["beta"]), EPS)
    by, bm, br = ref.ln_forward_bounds(d, ref.f64(c["gamma"]), ref.f64(c["beta"]), EPS, torch.float32)
    ref.within(y, yr, by, "y")
    ref.within(rstd, rr, br, "rstd")


def test_gradients_against_differences():
    """<grad, direction> against central differences of the float64 forward."""
    T, h = 19, 328
    c = draw(T, h, torch.float32, 8)
    g = {k: v.cuda() for k, v in c.items()}
    d = {k: ref.f64(v) for k, v in c.items()}
    _, mean, rstd = binding.tp_ln_forward(g["x"], g["gamma"], g["beta"], EPS)
    grads = binding.tp_ln_backward(g["dy"], g["x"], g["gamma"], mean, rstd)
    rng = np.random.default_rng(0)
    f = lambda x, ga, be: float((ref.ln_forward(x, ga, be, EPS)[0] * d["dy"]).sum())  # noqa: E731
    args = [d["x"], d["gamma"], d["beta"]]
    for i, grad in enumerate(grads):
        v = rng.standard_normal(args[i].shape)
        step = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * v, args[i] - step * v
        diff = (f(*up) - f(*down)) / (2 * step)
        got = float((ref.f64(grad) * v).sum())
        # the gradients' own error (about 2^-20 of their terms) and the
        # difference's (cubic term, cancellation): 1e-4 of the terms' size
        assert abs(got - diff) <= 1e-4 * np.linalg.norm(ref.f64(grad)) * np.sqrt(v.size) ** 0.5 + 1e-6


def test_rows_behind_the_last_stay():
    """Outputs that are the front of a larger buffer: the rest is not touched."""
    T, h = 13, 1023
    for dtype in TYPES:
        c = {k: v.cuda() for k, v in draw(T, h, dtype, 4).items()}
        y = torch.full((T + 3, h), 7.0, dtype=dtype, device="cuda")
        dx = torch.full((T + 3, h), 7.0, dtype=dtype, device="cuda")
        stats = [torch.full((T + 3,), 7.0, device="cuda") for _ in range(2)]
        _, mean, rstd = binding.tp_ln_forward(c["x"], c["gamma"], c["beta"], EPS, y=y[:T],
                                              mean=stats[0][:T], rstd=stats[1][:T])
        binding.tp_ln_backward(c["dy"], c["x"], c["gamma"], mean, rstd, dx=dx[:T])
        for t in (y, dx, *stats):
            assert bool((t[T:] == 7.0).all()) and not bool((t[:T] == 7.0).all())


@pytest.mark.parametrize("T,h", [(2048, 20480), (700, 1024), (300, 2047)])
def test_backward_is_deterministic(T, h):
    c = {k: v.cuda() for k, v in draw(T, h, torch.bfloat16, 11).items()}
    _, mean, rstd = binding.tp_ln_forward(c["x"], c["gamma"], c["beta"], EPS)
    first = binding.tp_ln_backward(c["dy"], c["x"], c["gamma"], mean, rstd)
    need = binding.lib().tp_ln_backward_workspace_floats(T, h, 0)
    dirty = torch.full((need,), float("nan"), device="cuda")
    for _ in range(3):
        again = binding.tp_ln_backward(c["dy"], c["x"], c["gamma"], mean, rstd, partial=dirty)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_empty_batch():
    for dtype in TYPES:
        e = torch.empty((0, 24), dtype=dtype, device="cuda")
        p = torch.ones(24, dtype=dtype, device="cuda")
        y, mean, rstd = binding.tp_ln_forward(e, p, p, EPS)
        dx, dg, db = binding.tp_ln_backward(e, e, p, mean, rstd, dgamma=torch.ones(24, device="cuda"),
                                            dbeta=torch.ones(24, device="cuda"))
        assert y.shape == (0, 24) and dx.shape == (0, 24)
        assert float(dg.abs().max()) == 0.0 and float(db.abs().max()) == 0.0


def test_captured_and_on_another_stream():
    """The calls captured into a graph and replayed on new inputs, and run on
    a stream that is not the current one, give the eager results."""
    T, h = 203, 1024
    a, b = (draw(T, h, torch.bfloat16, s) for s in (1, 2))
    s = {k: v.cuda() for k, v in a.items()}
    run = lambda st=None: binding.tp_ln_backward(  # noqa: E731
        s["dy"], s["x"], s["gamma"], *binding.tp_ln_forward(s["x"], s["gamma"], s["beta"], EPS, stream=st)[1:],
        stream=st)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for c in (b, a):
        for k, v in c.items():
            s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = run(side)
        raw = run(side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(other, want))
        assert all(torch.equal(p, q) for p, q in zip(raw, want))


def test_offsets_beyond_32_bits():
    """More than 2^31 values: a block of rows repeated, whose repeats must all
    come out alike; dgamma and dbeta are as many times the block's sums."""
    rows, h, times = 1000, 16384, 140
    c = draw(rows, h, torch.bfloat16, 12)
    g = {k: v.cuda() for k, v in c.items()}
    x, dy = g["x"].repeat(times, 1), g["dy"].repeat(times, 1)
    y, mean, rstd = binding.tp_ln_forward(x, g["gamma"], g["beta"], EPS)
    dx, dgamma, dbeta = binding.tp_ln_backward(dy, x, g["gamma"], mean, rstd)
    for t in (y, mean, rstd, dx):
        t = t.view(times, rows, -1)
        for i in range(1, times):
            assert torch.equal(t[i], t[0]), i
    d = {k: ref.f64(v) for k, v in c.items()}
    by, _, _ = ref.ln_forward_bounds(d["x"], d["gamma"], d["beta"], EPS, torch.bfloat16)
    ref.within(y[-rows:], ref.ln_forward(d["x"], d["gamma"], d["beta"], EPS)[0], by, "y")
    m, r = ref.f64(mean[:rows]), ref.f64(rstd[:rows])
    out = ref.ln_backward(d["dy"], d["x"], d["gamma"], m, r)
    bx, bg, bb = ref.ln_backward_bounds(d["dy"], d["x"], d["gamma"], m, r, torch.bfloat16)
    ref.within(dx[-rows:], out[0], bx, "dx")
    chains = (rows * times + 16) / (rows + 16)  # the sums' chains are longer
    ref.within(dgamma, times * out[1], times * chains * bg, "dgamma")
    ref.within(dbeta, times * out[2], times * chains * bb, "dbeta")
