"""The waits of the kernels, by themselves: each gives up after the time that it
is given, whether it counts time or polls, and the norm's calls leave the
status word alone."""

import time

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ms", [5, 100, 400])
def test_waits_give_up_in_their_time(ms):
    """The status word is written when the wait by time, its neighbour's and the
    wait by polls have all given up: not long before the limit (the timer
    ticks, polls differ by some percent), nor long behind it."""
    binding.selftest_bounded_wait(1000)  # the module is loaded
    torch.cuda.synchronize()
    t = time.perf_counter()
    status = binding.selftest_bounded_wait(1000 * ms)
    took = time.perf_counter() - t
    assert status == binding.TPMLP_ERR_DEVICE_TIMEOUT
    assert 0.7e-3 * ms <= took <= 2e-3 * ms + 0.2, took
    assert binding.device_status() == binding.TPMLP_OK


@pytest.mark.parametrize("T,h", [(5, 64), (700, 1024), (300, 8192), (77, 1023), (3, 65544)])
def test_the_norm_leaves_the_status_word(T, h):
    assert binding.device_status() == binding.TPMLP_OK
    x, p = torch.randn(T, h, device="cuda"), torch.ones(h, device="cuda")
    _, mean, rstd = binding.tp_ln_forward(x, p, p)
    binding.tp_ln_backward(x, x, p, mean, rstd)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.TPMLP_OK
