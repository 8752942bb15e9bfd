"""The calls around the experts (moe_layer_few, moe_layer_norm, moe_linear, block.py) at the edges of their arguments, on
the host."""
import pytest

from routing_permute_groupgemm_amd import _lib, block, synth


@pytest.mark.parametrize("Kd,N", [(64, 64), (2048, 64), (2112, 64), (7168, 2048), (2048, 7168), (1 << 21, 64)])
def test_plans_of_the_dense_product_without_rows(Kd, N):
    """moe_linear_backward of no rows still writes dw and db, so its size function is asked."""
    assert _lib.moe_linear_workspace_size(0, Kd, N) == 0
    assert _lib.moe_linear_backward_workspace_size(0, Kd, N) == 0


def test_block_of_no_tokens_is_allocated():
    shape = synth.WORKLOADS["tiny"].scaled(T=0, H=192, F=128, E=64, K=3, backward=True)
    b = block.BlockBuffers.allocate(shape, shared=2112, device="cpu")
    assert b.out.shape == (0, 192) and b.grads["shared_down"].shape == (1, 2112, 192)
