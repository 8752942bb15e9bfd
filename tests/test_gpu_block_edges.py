"""The calls around the experts at the edges of their arguments."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, block
from test_gpu_block import SHAPE, weights

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(seed, *shape, std=1.0, dtype=BF):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("Kd,N", [(2112, 64), (7168, 2048), (2048, 4160)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_dense_backward_without_rows(Kd, N, act):
    """No rows: zeros in dw and db, for long contractions too."""
    x, dy, w = rand(1, 0, Kd), rand(2, 0, N), rand(3, Kd, N)
    dw, db = torch.full((Kd, N), 5.0, device="cuda"), torch.full((N,), 5.0, device="cuda")
    print(f"[linear] no rows, {Kd} x {N} {act}", flush=True)
    dz, dx, _, _ = _lib.moe_linear_backward(dy, x, w, act=act, z=None if act == "none" else dy, dw=dw, db=db)
    assert dz.shape == (0, N) and dx.shape == (0, Kd) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shared", [0, 64])
def test_block_returns_what_it_has_written(rms, shared):
    """Every gradient that the backward returns is of a weight that there is (or of x), and is written."""
    T = 5
    shape, p = SHAPE.scaled(T=T), weights(SHAPE, shared, rms)
    b = block.BlockBuffers.allocate(shape, shared=shared)
    for buf in b.grads.values():
        buf.fill_(float("nan"))
    x, d = rand(1, T, 192), rand(2, T, 192)
    block.forward(b, p, x, rand(3, T, 192))
    g = block.backward(b, p, d)
    assert set(g) <= set(p) | {"x"} and ("norm_bias" in g) == (not rms)
    for name, grad in g.items():
        assert torch.isfinite(grad).all(), name


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shared", [0, 2112])
def test_block_of_no_tokens(rms, shared):
    """An empty batch: no rows out, and the weights' gradients are zeros."""
    shape, p = SHAPE.scaled(T=0), weights(SHAPE, shared, rms)
    b = block.BlockBuffers.allocate(shape, shared=shared)
    for buf in b.grads.values():
        buf.fill_(5.0)
    x = rand(1, 0, 192)
    s, out = block.forward(b, p, x, x)
    assert s.shape == out.shape == (0, 192)
    for name, grad in block.backward(b, p, x, x).items():
        assert (grad == 0).all(), name
