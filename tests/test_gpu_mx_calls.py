"""Calls of the block-scaled operators that moe.h allows at the edges of their arguments."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib

pytestmark = pytest.mark.gpu


def normal(seed, *shape, std=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


@pytest.mark.parametrize("rows", [1, 70])
def test_combine_without_tokens_writes_the_rows(rows):
    """No token (an empty batch beside rows of other GPUs): y is moe_grouped_gemm4's, which rounds the same sums."""
    a, w = normal(1, rows, 192), _lib.moe_pack4(normal(2, 2, 192, 128, std=0.05))
    offsets = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    y = torch.full((rows + 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    out = _lib.moe_grouped_gemm4_combine(a, w, offsets, rows, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                                         torch.empty((0, 2), device="cuda"), y=y)
    assert out.shape == (0, 128)
    assert torch.equal(y[:rows], _lib.moe_grouped_gemm4(a, w, offsets, rows)) and (y[rows:] == 5.0).all()
