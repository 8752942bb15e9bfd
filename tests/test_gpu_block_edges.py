"""The calls around the experts at the edges of their arguments."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, block
from test_gpu_block import SHAPE, near, reference, weights

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


@pytest.mark.parametrize("T,EL", [(1, 64), (37, 64), (700, 24)])
def test_block_gradient_of_the_router_bias(T, EL):
    """The scores' bias against autograd in 64 bits, with as many roundings in line as the router's weights; without a bias
    there is no gradient of one, and the others keep their bits."""
    shape = SHAPE.scaled(T=T, e_local=EL, e_begin=0 if EL == 64 else 8)
    p = weights(shape, 64, False)
    b = block.BlockBuffers.allocate(shape, shared=64)
    x, d_out = rand(20, T, 192, std=1.5), rand(22, T, 192)
    block.forward(b, p, x)
    g = block.backward(b, p, d_out)
    assert set(g) == set(p) | {"x"}
    ref = {k: v.double().requires_grad_() for k, v in p.items()}
    out = reference(ref, x.double(), None, b.layer.topk_idx.long(), shape.e_begin)[1]
    (out * d_out.double()).sum().backward()
    near("router_bias", g["router_bias"], ref["router_bias"].grad, 10)
    p["router_bias"].zero_()
    block.forward(b, p, x)
    want = {k: v.clone() for k, v in block.backward(b, p, d_out).items()}
    p["router_bias"] = None
    block.forward(b, p, x)
    got = block.backward(b, p, d_out)
    assert set(got) == set(want) - {"router_bias"}
    for k in got:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("T,E", [(1, 64), (4, 192), (32, 320), (33, 64), (1000, 256), (4099, 4096), (70001, 128)])
def test_router_bias_backward(T, E):
    """Whole numbers bit for bit, so no row or column is left out or taken twice; values against 64 bits, at most T
    additions on any path; the caller's workspace, what is behind it, and the same bits again."""
    F32 = torch.float32
    print(f"[router bias] T={T} E={E}", flush=True)
    whole = torch.randint(-9, 10, (T, E), device="cuda").to(F32)
    assert torch.equal(_lib.moe_router_bias_backward(whole).double(), whole.double().sum(0))
    d = rand(T + E, T, E, dtype=F32)
    got = _lib.moe_router_bias_backward(d)
    assert ((got.double() - d.double().sum(0)).abs() <= T * 2.0 ** -24 * d.double().abs().sum(0)).all()
    n = _lib.moe_router_bias_backward_workspace_size(T, E)
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.empty(E, device="cuda")
    assert _lib.moe_router_bias_backward(d, dbias=out, ws=ws) is out and torch.equal(out, got) and (ws[n:] == 0xA5).all()


def test_router_bias_backward_at_its_edges():
    out = torch.full((128,), 5.0, device="cuda")
    assert (_lib.moe_router_bias_backward(torch.empty((0, 128), device="cuda"), dbias=out) == 0).all()
    d = torch.zeros((5, 128), device="cuda")
    d[3, 7], d[2, 9] = float("nan"), float("inf")
    got = _lib.moe_router_bias_backward(d)
    assert torch.isnan(got[7]) and torch.isposinf(got[9]) and int((got == 0).sum()) == 126
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d = rand(3, 600, 128, dtype=torch.float32)
    got = _lib.moe_router_bias_backward(d, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, _lib.moe_router_bias_backward(d))
    for kw in (dict(dlogits=d.double()), dict(dlogits=d.t()), dict(dlogits=d[0]), dict(dlogits=d[:, :96].contiguous()),
               dict(dbias=out[:64]), dict(dbias=out.double()), dict(ws=out)):
        with pytest.raises(_lib.MoeError):
            _lib.moe_router_bias_backward(**dict(dict(dlogits=d), **kw))


def test_block_on_a_share_that_every_token_chooses():
    """More rows than twice the expected: dropped and said so at the default capacity; with room for every pair, or in the
    few-token form, the output of all of them."""
    T = 6
    shape = SHAPE.scaled(T=T, e_local=8, e_begin=16, backward=False)
    p = weights(shape, 64, True)
    p["router_bias"][16:24] += 50.0
    x = rand(5, T, 192)
    ref = {k: v.double() for k, v in p.items()}
    b = block.BlockBuffers.allocate(shape, shared=64)
    block.forward(b, p, x)
    assert b.layer.cap < 3 * T and int(b.layer.status[0]) == 1
    for kw in (dict(cap=3 * T), dict(few=True)):
        b = block.BlockBuffers.allocate(shape, shared=64, **kw)
        s, out = block.forward(b, p, x)
        assert kw.get("few") or int(b.layer.status[0]) == 0
        near("out", out, reference(ref, s.double(), None, b.layer.topk_idx.long(), 16)[1], 4)
    with pytest.raises(_lib.MoeError):
        block.BlockBuffers.allocate(shape, few=True, cap=3 * T)
