"""Scratch sizes and refusals of the output head and the final norm at the ends
of their ranges, on a host without a GPU."""

import pytest

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
