"""The scratch of packed attention and of the norms and rotation over all batches, on a
host without a GPU."""

import pytest

from tensor_transformer_mlp_forward_gb300 import binding, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def _base(nb, T, nh):
    """The plan and delta."""
    return 16 * (T // 128 + nb) + 4 * (T // 128 + 2) + 4 * T * nh + 2048


@pytest.mark.parametrize("nkv", [1, 2, 3, 4, 8, 16])
@pytest.mark.parametrize("group", [2, 3, 4, 5, 7, 8, 13, 16, 17, 71, 113])
def test_parts_scratch_is_bounded_for_every_group(L, group, nkv):
    # the parts' fp32 sums: at most 2 * 228 * 128 rows of dK and dV
    d = 160
    for tiles in sorted({1, 2, 7, 30, 57, 75, 76, 113, 114, 200, 226, 227, 228, 300}):
        for T in (128 * (tiles // nkv + 1) - 1, 128 * max(tiles // nkv, 1)):
            for nb in (1, 2, 30):
                need = L.tp_attn_packed_backward_workspace_bytes(nb, T, group * nkv, nkv, d)
                assert need <= _base(nb, T, group * nkv) + 2 * 228 * 128 * 2 * d * 4, (nb, T)


@pytest.mark.parametrize("nb", [0, 1, 2, 9])
def test_scratch_of_no_tokens(L, nb):
    assert 0 < L.tp_attn_packed_backward_workspace_bytes(nb, 0, 8, 2, 128) < 1 << 20
    assert 0 < L.tp_attn_packed_forward_workspace_bytes(nb, 0, 8, 2, 128) < 1 << 20
    assert L.tp_qk_norm_rope_backward_workspace_floats(0, 8, 2, 128) == 0


@pytest.mark.parametrize("nh,nkv,d", [(16, 4, 160), (32, 8, 128), (16, 1, 64), (28, 4, 128), (71, 1, 64), (20, 20, 64),
                                      (456, 228, 64), (454, 227, 64)])
def test_scratch_never_shrinks_with_the_batch(L, nh, nkv, d):
    # a program that sizes its scratch for its largest batch may run any smaller one
    Ts = sorted({0, 1, 127, 128, 129, 1000, 2000, 3585, 5000, 6007, 7295, 7296, 7297, 8191, 8192, 14591, 14592, 14593,
                 29055, 29056, 29057, 29183, 29184, 29185, 40000, 1 << 17, 1 << 20})
    nbs = [1, 2, 3, 7, 10, 23, 57, 100, 300, 455, 456, 457, 5000]
    for f in (lambda nb, T: L.tp_attn_packed_forward_workspace_bytes(nb, T, nh, nkv, d),
              lambda nb, T: L.tp_attn_packed_backward_workspace_bytes(nb, T, nh, nkv, d)):
        for nb in nbs:
            sizes = [f(nb, T) for T in Ts]
            assert sizes == sorted(sizes), nb
        for T in Ts:
            sizes = [f(nb, T) for nb in nbs]
            assert sizes == sorted(sizes), T
    sizes = [L.tp_qk_norm_rope_backward_workspace_floats(T, nh, nkv, d) for T in Ts]
    assert sizes == sorted(sizes)
