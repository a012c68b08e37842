"""Scratch sizes and refusals of the output head and the final norm at the ends
of their ranges, on a host without a GPU."""

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("T", [1, 7, 8, 9, 16])
def test_few_tokens_keep_no_logits_where_one_kernel_does_all(L, T):
    """Rows of up to 1024 values: dX's planes, at most 304 [T, h] of fp32, and
    nothing that grows with the vocabulary."""
    for h in (8, 512, 1024):
        sizes = {V: L.tp_head_loss_backward_workspace_bytes(T, h, V) for V in (50257, 131072, 1 << 30)}
        assert len(set(sizes.values())) == 1, sizes
        assert sizes[50257] <= 512 + 304 * 4 * T * h
        assert L.tp_head_loss_backward_min_workspace_bytes(T, h, 50257) == sizes[50257]
    # wider rows keep the logits' gradient of 16 tokens twice
    assert L.tp_head_loss_backward_workspace_bytes(T, 1032, 50257) >= 2 * 2 * 16 * 50257


def test_rows_wider_than_the_kernels_count(L):
    """h = 2^31 - 8: a column counter behind the row's end would pass 2^31 (the
    few-token kernels would see no column at all).  2^30 is the widest."""
    import ctypes

    P, N = ctypes.c_void_p(0x10000), None
    big = ctypes.c_size_t(1 << 62)
    for h in ((1 << 31) - 8, (1 << 30) + 8):
        assert L.tp_head_loss_forward(P, P, P, 1, h, 5, P, P, P, big, N) == binding.TPMLP_ERR_SHAPE
        assert L.tp_head_loss_backward(P, P, P, P, P, 1, h, 5, P, P, P, big, N) == binding.TPMLP_ERR_SHAPE
        assert L.tp_head_loss_forward_workspace_bytes(1, h, 5) == 0
        assert L.tp_head_loss_backward_workspace_bytes(1, h, 5) == 0
    assert L.tp_head_loss_forward_workspace_bytes(1, 1 << 30, 5) > 0
    assert L.tp_head_loss_backward_workspace_bytes(1, 1 << 30, 5) > 0


def test_sizes_beyond_32_bits_are_refused():
    """A row count that 32 bits cut to another (2^32 + 4 to 4) is no call of four
    rows.  Tensors without memory: their shapes are answered first."""
    n = (1 << 32) + 4
    m = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    for T, h in ((n, 1), (1 << 31, 1), ((1 << 30) + 1, 1), (1, n)):
        x, p, stat = m(T, h), m(h), m(T, dtype=torch.float32)
        with pytest.raises(ValueError, match="at most 2.30"):
            binding.tp_ln_forward(x, p, p)
        with pytest.raises(ValueError, match="at most 2.30"):
            binding.tp_ln_backward(x, x, p, stat, stat)
    for T, h, V in ((n, 8, 5), (4, n + 4, 5), (4, 8, n)):
        X, W, y, f = m(T, h), m(V, h), m(T, dtype=torch.int64), m(T, dtype=torch.float32)
        with pytest.raises(ValueError, match="at most 2.30"):
            binding.tp_head_loss_forward(X, W, y)
        with pytest.raises(ValueError, match="at most 2.30"):
            binding.tp_head_loss_backward(f, X, W, y, f)
        for size in (binding.head_loss_backward_workspace_bytes, binding.head_loss_backward_min_workspace_bytes):
            with pytest.raises(ValueError, match="at most 2.30"):
                size(T, h, V)
