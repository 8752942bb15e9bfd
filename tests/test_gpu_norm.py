"""Layer norm, forward and backward, against its formula in 64 bits and against differences."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative


def rand(seed, *shape, std=1.0, shift=0.0, dtype=F32):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std + shift).to(dtype)


def step(dtype):
    return 2.0 ** -8 if dtype == BF else U


def stats(s, eps, rms):
    s = s.double()
    mean = torch.zeros_like(s[:, :1]) if rms else s.mean(1, keepdim=True)
    return s, mean, 1 / ((s - mean).square().mean(1, keepdim=True) + eps).sqrt()


SHAPES = [(1, 64), (3, 64), (2, 128), (5, 448), (7, 512), (300, 576), (33, 1024), (1, 2048), (400, 2048), (19, 2112),
          (500, 2112), (1, 7168), (300, 7168), (4, 8192), (290, 8192), (2, 8256), (270, 8256), (1, 16384), (259, 16384),
          # one row a CU and one more, and passes that go past the caches
          (256, 1024), (257, 1024), (9001, 2048), (3001, 7168)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rms", [False, True])
def test_forward(T, H, dtype, rms):
    """Sums of a thread's at most 32 values, a wave and 16 waves: at most 64 roundings on any path, so 128 U covers the
    mean's correction, the spread and the quotient together; the output is rounded once."""
    x = rand(T + H, T, H, std=3.0, shift=0.7, dtype=dtype)
    add = rand(1, T, H, dtype=BF)
    weight, bias = rand(2, H, std=0.3, shift=1.0), None if rms else rand(3, H)
    print(f"[norm] T={T} H={H} {dtype} rms={rms}", flush=True)
    s, y, mean, rstd = _lib.moe_layer_norm(x, weight, bias, add=add, rms=rms)
    assert torch.equal(s, (x.float() + add.float()).to(dtype))
    v, m, r = stats(s, 1e-5, rms)
    xh, spread = (v - m) * r, (v - m).abs().mean(1, keepdim=True)
    assert ((rstd.double() - r[:, 0]).abs() <= 128 * U * r[:, 0]).all()
    if rms:
        assert mean is None
    else:
        assert ((mean.double() - m[:, 0]).abs() <= 128 * U * spread[:, 0] + 2 * U * m[:, 0].abs()).all()
    want = xh * weight.double() + (0 if rms else bias.double())
    tol = 2.0 ** -8 * want.abs() + 128 * U * (weight.abs() * (xh.abs() + r * spread) + (0 if rms else bias.abs()))
    assert ((y.double() - want).abs() <= 1.01 * tol).all()


@pytest.mark.parametrize("rms", [False, True])
def test_forward_without_the_options(rms):
    """No addition, weight or bias; buffers of the caller's, the sum in place."""
    x = rand(1, 9, 320, std=2.0, dtype=BF)
    s, y, mean, rstd = _lib.moe_layer_norm(x, rms=rms, eps=0.0)
    assert s is x
    v, m, r = stats(x, 0.0, rms)
    want = (v - m) * r
    assert ((y.double() - want).abs() <= 1.01 * (2.0 ** -8 * want.abs() + 128 * U * (want.abs() + 1))).all()
    ones, zeros = torch.ones(320, device="cuda"), torch.zeros(320, device="cuda")
    assert torch.equal(_lib.moe_layer_norm(x, ones, zeros, rms=rms, eps=0.0)[1], y)
    add = rand(2, 9, 320, dtype=BF)
    want = _lib.moe_layer_norm(x, add=add, rms=rms)
    stream = x.clone()
    got = _lib.moe_layer_norm(stream, add=add, rms=rms, sum=stream, y=torch.empty_like(y), rstd=torch.empty_like(rstd))
    assert got[0] is stream
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a, b)
    copy = torch.empty_like(x)
    assert torch.equal(_lib.moe_layer_norm(x, rms=rms, sum=copy)[0], x) and torch.equal(copy, x)


def test_offset_that_is_large_against_the_spread():
    """Mean 10^4, spread 1: the mean's own rounding in fp32 (10^-3) would show in every value."""
    x = rand(5, 40, 4096, shift=1e4)
    _, y, mean, rstd = _lib.moe_layer_norm(x)
    v, m, r = stats(x, 1e-5, False)
    xh = (v - m) * r
    assert ((y.double() - xh).abs() <= 1.01 * (2.0 ** -8 * xh.abs() + 128 * U * (xh.abs() + 1))).all()
    assert ((rstd.double() - r[:, 0]).abs() <= 128 * U * r[:, 0]).all()
    assert ((mean.double() - m[:, 0]).abs() <= 128 * U + 2 * U * 1.01e4).all()


def test_rows_of_one_value_of_nan_and_of_infinity():
    x = torch.full((5, 192), 3.0, dtype=BF, device="cuda")
    x[1], x[2, 7], x[3, 9] = 0.0, float("nan"), float("inf")
    x[4] = rand(1, 192, dtype=BF)
    _, y, mean, rstd = _lib.moe_layer_norm(x)
    assert (y[:2] == 0).all() and torch.isfinite(rstd[:2]).all()
    assert ((rstd[:2].double() * 1e-5 ** 0.5 - 1).abs() <= 64 * U).all()
    assert torch.isnan(y[2]).all() and torch.isnan(rstd[2]) and torch.isnan(y[3]).all() and torch.isnan(rstd[3])
    assert torch.equal(y[4:], _lib.moe_layer_norm(x[4:].contiguous())[1])
    _, y, _, rstd = _lib.moe_layer_norm(x, rms=True)
    assert torch.isnan(y[2]).all() and torch.isnan(rstd[2]) and rstd[3] == 0 and torch.isnan(y[3, 9])


@pytest.mark.parametrize("T,H", SHAPES + [(5000, 192), (1100, 2048)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rms", [False, True])
def test_backward(T, H, dtype, rms):
    """From the same fp32 mean and rstd in 64 bits: sums over a row as in the forward; over the rows at most T + 32
    additions on any path."""
    s = rand(T * 3 + H, T, H, std=2.0, shift=0.5, dtype=dtype)
    dy, d_sum = rand(7, T, H, dtype=BF), rand(8, T, H, dtype=dtype)
    weight = rand(9, H, std=0.3, shift=1.0)
    mean, rstd = (a[:, 0].float() for a in stats(s, 1e-5, rms)[1:])
    print(f"[norm] backward T={T} H={H} {dtype} rms={rms}", flush=True)
    dx, dw, db = _lib.moe_layer_norm_backward(dy, s, weight, None if rms else mean, rstd, d_sum=d_sum, rms=rms)
    r = rstd.double()[:, None]
    xh = (s.double() - (0 if rms else mean.double()[:, None])) * r
    g = dy.double() * weight.double()
    c1, c2 = (torch.zeros_like(r) if rms else g.mean(1, keepdim=True)), (g * xh).mean(1, keepdim=True)
    want = r * (g - c1 - xh * c2) + d_sum.double()
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + d_sum.abs()
    assert dx.dtype == dtype
    assert ((dx.double() - want).abs() <= 1.01 * (step(dtype) * want.abs() + 128 * U * size)).all()
    terms = dy.double() * xh
    assert ((dw.double() - terms.sum(0)).abs() <= (T + 36) * U * terms.abs().sum(0)).all()
    if rms:
        assert db is None
    else:
        assert ((db.double() - dy.double().sum(0)).abs() <= (T + 32) * U * dy.double().abs().sum(0)).all()
    # the same bits again, and with the gradients' buffers left out
    again = _lib.moe_layer_norm_backward(dy, s, weight, mean, rstd, d_sum=d_sum, rms=rms, want_db=False)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and again[2] is None
    again = _lib.moe_layer_norm_backward(dy, s, weight, mean, rstd, d_sum=d_sum, rms=rms, want_dw=False)
    assert torch.equal(again[0], dx) and again[1] is None and (rms or torch.equal(again[2], db))
    alone = _lib.moe_layer_norm_backward(dy, s, weight, mean, rstd, d_sum=d_sum, rms=rms, want_dw=False, want_db=False)
    assert torch.equal(alone[0], dx) and alone[1] is None and alone[2] is None


@pytest.mark.parametrize("rms", [False, True])
def test_backward_without_weight_and_residual_and_in_place(rms):
    s, dy = rand(1, 6, 640, dtype=BF), rand(2, 6, 640, dtype=BF)
    _, _, mean, rstd = _lib.moe_layer_norm(s, rms=rms)
    dx = _lib.moe_layer_norm_backward(dy, s, None, mean, rstd, rms=rms)[0]
    ones, zeros = torch.ones(640, device="cuda"), torch.zeros((6, 640), dtype=BF, device="cuda")
    assert torch.equal(dx, _lib.moe_layer_norm_backward(dy, s, ones, mean, rstd, d_sum=zeros, rms=rms)[0])
    d_sum = rand(3, 6, 640, dtype=BF)
    want = _lib.moe_layer_norm_backward(dy, s, None, mean, rstd, d_sum=d_sum, rms=rms)[0]
    got = _lib.moe_layer_norm_backward(dy, s, None, mean, rstd, d_sum=d_sum, rms=rms, dx=d_sum)[0]
    assert got is d_sum and torch.equal(got, want)


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_against_differences(rms):
    """Central differences in 64 bits of L = sum(dy * y): step 10^-4 on values of order 1 leaves about 10^-8 of L's
    scale, below the kernel's fp32 roundings (128 U of the terms' sizes)."""
    T, H, h = 4, 192, 1e-4
    s, dy = rand(21, T, H, std=1.5, shift=0.4), rand(22, T, H, dtype=BF)
    weight, bias = rand(23, H, std=0.3, shift=1.0), rand(24, H)
    _, _, mean, rstd = _lib.moe_layer_norm(s, weight, None if rms else bias, rms=rms)
    dx, dw, db = _lib.moe_layer_norm_backward(dy, s, weight, mean, rstd, rms=rms)

    def loss(s, w, b):
        _, m, r = stats(s, 1e-5, rms)
        return (dy.double() * ((s - m) * r * w + b)).sum()

    s64, w64, b64 = s.double(), weight.double(), torch.zeros_like(bias.double()) if rms else bias.double()
    for i, grad in enumerate((dx, dw, db)):
        if grad is None:
            continue
        at = [s64, w64, b64]
        v = rand(30 + i, *at[i].shape).double()
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = (grad.double() * v).sum()
        assert abs(float(diff - got)) <= 1e-6 * float((grad.double() * v).abs().sum()) + 1e-6


def test_no_tokens():
    x = torch.empty((0, 128), dtype=BF, device="cuda")
    s, y, mean, rstd = _lib.moe_layer_norm(x)
    assert y.shape == (0, 128) and mean.shape == rstd.shape == (0,)
    dw, db = torch.full((128,), 5.0, device="cuda"), torch.full((128,), 5.0, device="cuda")
    dx, _, _ = _lib.moe_layer_norm_backward(x, x, None, mean, rstd, dw=dw, db=db)
    assert dx.shape == (0, 128) and (dw == 0).all() and (db == 0).all()


def test_rows_past_2_31_values():
    """Offsets past 32 bits: 2^31 / 16384 rows and some, checked at both ends and around the border."""
    T, H = (1 << 17) + 5, 16384
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    probe = [0, 1, (1 << 16) - 1, 1 << 16, (1 << 17) - 1, 1 << 17, T - 1]
    rows = rand(41, len(probe), H, dtype=BF)
    x[probe] = rows
    print(f"[norm] {T} x {H}", flush=True)
    y, mean, rstd = _lib.moe_layer_norm(x)[1:]
    want = _lib.moe_layer_norm(rows)
    v, m, r = stats(rows, 1e-5, False)
    ref = (v - m) * r
    for got in (y[probe], want[1]):
        assert ((got.double() - ref).abs() <= 1.01 * (2.0 ** -8 * ref.abs() + 128 * U * (ref.abs() + 1))).all()
    del y
    dx, dw, db = _lib.moe_layer_norm_backward(x, x, None, mean, rstd)
    g, c = v, v.mean(1, keepdim=True)
    back = r * (g - c - ref * (g * ref).mean(1, keepdim=True))
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + ref.abs() * (g * ref).abs().mean(1, keepdim=True))
    assert ((dx[probe].double() - back).abs() <= 1.01 * (2.0 ** -8 * back.abs() + 160 * U * size)).all()
    assert ((dw.double() - (v * ref).sum(0)).abs() <= (T + 64) * U * (v * ref).abs().sum(0)).all()
    assert ((db.double() - v.sum(0)).abs() <= (T + 64) * U * v.abs().sum(0)).all()


def test_refusals():
    x, w = rand(1, 4, 128, dtype=BF), rand(2, 128)
    for kw in (dict(weight=w[:64].contiguous()), dict(weight=w.to(BF)), dict(add=x.float()), dict(add=x[:2].contiguous()),
               dict(y=x.float()), dict(eps=-1.0), dict(eps=float("nan")), dict(rms=True, mean=w[:4].contiguous()),
               dict(sum=x.float()), dict(rstd=w)):
        with pytest.raises(_lib.MoeError):
            _lib.moe_layer_norm(x, **kw)
    for bad in (x.half(), x.t(), x[0], rand(3, 4, 96, dtype=BF), rand(3, 4, 16448, dtype=BF)):
        with pytest.raises(_lib.MoeError):
            _lib.moe_layer_norm(bad)
    _, _, mean, rstd = _lib.moe_layer_norm(x)
    for args, kw in (((x, x, w, None, rstd), {}), ((x, x, w, mean, None), {}), ((x, x, w, None, rstd), dict(rms=True, want_db=True)),
                     ((x.float(), x, w, mean, rstd), {}), ((x, x, w, mean, rstd), dict(d_sum=x.float())),
                     ((x, x.float(), w, mean, rstd), dict(dx=x)), ((x[:3].contiguous(), x, w, mean, rstd), {})):
        with pytest.raises(_lib.MoeError):
            _lib.moe_layer_norm_backward(*args, **kw)
