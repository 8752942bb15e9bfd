"""The calls around the experts at the edges of their arguments."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib

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
