"""The dense product with bias, activation and residual, forward and backward, against its formula in 64 bits."""
import math

import pytest
import torch

from routing_permute_groupgemm_amd import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu"]


def rand(seed, *shape, std=1.0, dtype=F32):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def ints(seed, *shape, top=2, dtype=BF):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").to(dtype)


def act64(act, z):
    return {"none": z, "relu": z.clamp(min=0), "silu": z * torch.sigmoid(z),
            "gelu": 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))}[act]


def slope64(act, z):
    s = torch.sigmoid(z)
    return {"none": torch.ones_like(z), "relu": (z > 0).double(), "silu": s * (1 + z * (1 - s)),
            "gelu": 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[act]


# each form: a few rows (one chunk of the contraction and several), small tiles with and without chunks, large tiles;
# rows and columns that fill no tile
SHAPES = [(1, 64, 64), (1, 2048, 7168), (2, 64, 192), (15, 512, 320), (16, 1088, 128), (17, 4096, 64), (32, 256, 1536),
          (33, 320, 192), (41, 4096, 1536), (64, 192, 4160), (64, 64, 576), (65, 64, 64), (65, 2048, 320), (200, 7168, 256),
          (130, 192, 2112), (700, 1536, 832), (1000, 64, 4096), (4001, 2048, 768), (8200, 128, 2112), (16400, 64, 320),
          (4000, 4096, 4032)]


@pytest.mark.parametrize("T,Kd,N", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(T, Kd, N, act):
    """fp32 sums of Kd products (and the bias) in some order, slopes of at most 1.13, the activations' own functions
    within 2^-18 of their terms, one rounding to bf16 (z is rounded on its own)."""
    x, w = rand(T + Kd, T, Kd, dtype=BF), rand(N, Kd, N, std=0.05, dtype=BF)
    bias, res = rand(3, N), rand(4, T, N, dtype=BF)
    print(f"[linear] T={T} Kd={Kd} N={N} {act}", flush=True)
    y, z = _lib.moe_linear(x, w, bias=bias, act=act, residual=res, want_z=True)
    want = x.double() @ w.double() + bias.double()
    ez = (Kd + 8) * U * (x.double().abs() @ w.double().abs() + bias.double().abs())
    assert ((z.double() - want).abs() <= ez + 2.0 ** -8 * (want.abs() + ez) + 1e-37).all()
    a = act64(act, want)
    tol = 1.13 * ez + (2.0 ** -18 if act in ("silu", "gelu") else 0) * want.abs() + 2 * U * res.double().abs()
    a = a + res.double()
    assert ((y.double() - a).abs() <= tol + 2.0 ** -8 * (a.abs() + tol) + 1e-37).all()
    # without the options: the same sums
    plain, none = _lib.moe_linear(x, w)
    assert none is None
    want = want - bias.double()
    assert ((plain.double() - want).abs() <= ez + 2.0 ** -8 * (want.abs() + ez) + 1e-37).all()
    # the residual in place, the same bits again
    acc = res.clone()
    again, _ = _lib.moe_linear(x, w, bias=bias, act=act, residual=acc, y=acc)
    assert again is acc and torch.equal(acc, y)


# streamed rows, chunks, the three tiles, the largest with whole tiles alone and not
OPTIONS = [(40, 128, 192), (300, 4096, 320), (1000, 64, 4096), (2000, 2048, 4032), (4000, 128, 4160), (4096, 128, 4096)]


@pytest.mark.parametrize("T,Kd,N", OPTIONS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("with_bias", [False, True])
def test_every_set_of_options(T, Kd, N, act, with_bias):
    """Whether z is wanted changes no bit of y, whether there is a residual none of z; without an activation and a
    residual y is z; and y without a residual against float64, as above."""
    x, w = rand(T, T, Kd, dtype=BF), rand(N + 1, Kd, N, std=0.05, dtype=BF)
    bias, res = rand(3, N) if with_bias else None, rand(4, T, N, dtype=BF)
    print(f"[linear] options T={T} Kd={Kd} N={N} {act} bias {with_bias}", flush=True)
    y_res, z = _lib.moe_linear(x, w, bias=bias, act=act, residual=res, want_z=True)
    assert torch.equal(_lib.moe_linear(x, w, bias=bias, act=act, residual=res)[0], y_res)
    y, z_too = _lib.moe_linear(x, w, bias=bias, act=act, want_z=True)
    assert torch.equal(z_too, z)
    assert torch.equal(_lib.moe_linear(x, w, bias=bias, act=act)[0], y)
    want = x.double() @ w.double()
    ez = (Kd + 8) * U * (x.double().abs() @ w.double().abs())
    if with_bias:
        want += bias.double()
        ez += (Kd + 8) * U * bias.double().abs()
    if act == "none":
        assert torch.equal(y, z)
    tol = 1.13 * ez + (2.0 ** -18 if act in ("silu", "gelu") else 0) * want.abs()
    a = act64(act, want)
    assert ((y.double() - a).abs() <= tol + 2.0 ** -8 * (a.abs() + tol) + 1e-37).all()
    tol, a = tol + 2 * U * res.double().abs(), a + res.double()
    assert ((y_res.double() - a).abs() <= tol + 2.0 ** -8 * (a.abs() + tol) + 1e-37).all()


@pytest.mark.parametrize("T,Kd,N", SHAPES)
def test_exact_on_integers(T, Kd, N):
    """Whole numbers whose sums are exact in fp32 in any order: every output bit for bit, so no row, column or
    contraction step is taken twice, skipped or read from elsewhere."""
    x, w = ints(1, T, Kd), ints(2, Kd, N)
    bias, res, dy = ints(3, N, top=50, dtype=F32), ints(4, T, N, top=60), ints(5, T, N, top=1)
    print(f"[linear] integers T={T} Kd={Kd} N={N}", flush=True)
    y, z = _lib.moe_linear(x, w, bias=bias, act="relu", residual=res, want_z=True)
    want = x.double() @ w.double() + bias.double()
    assert torch.equal(z, want.float().to(BF))
    assert torch.equal(y, (want.clamp(min=0) + res.double()).float().to(BF))
    assert torch.equal(_lib.moe_linear(x, w)[0], (want - bias.double()).float().to(BF))
    for act in ("none", "relu"):
        dz, dx, dw, db = _lib.moe_linear_backward(dy, x, w, act=act, z=None if act == "none" else z)
        d = dy.double() if act == "none" else dy.double() * (z > 0)
        assert dz is dy if act == "none" else torch.equal(dz, d.to(BF))
        assert torch.equal(dx, (d @ w.double().t().contiguous()).float().to(BF))
        assert torch.equal(dw.double(), x.double().t().contiguous() @ d)
        assert torch.equal(db.double(), d.sum(0))


@pytest.mark.parametrize("T,Kd,N", [(1, 64, 64), (3, 128, 704), (64, 320, 192), (67, 192, 512), (700, 256, 576),
                                    (4001, 512, 768)])
@pytest.mark.parametrize("act", ACTS)
def test_backward(T, Kd, N, act):
    """dz rounds once; dx is the product of the rounded dz (its sums, its rounding), dw too; db sums before dz is
    rounded, at most T additions on any path.  The slopes are within 2^-18 of their terms."""
    x, w, dy = rand(1, T, Kd, dtype=BF), rand(2, Kd, N, std=0.05, dtype=BF), rand(3, T, N, dtype=BF)
    z = None if act == "none" else rand(4, T, N, std=1.5, dtype=BF)
    print(f"[linear] backward T={T} Kd={Kd} N={N} {act}", flush=True)
    dz, dx, dw, db = _lib.moe_linear_backward(dy, x, w, act=act, z=z)
    d = dy.double()
    e = torch.zeros_like(d)
    if act == "none":
        assert dz is dy
    else:
        v = z.double()
        d = dy.double() * slope64(act, v)
        e = (2.0 ** -18 if act in ("silu", "gelu") else 0) * dy.double().abs() * (1 + v.abs())
        assert ((dz.double() - d).abs() <= e + 2.0 ** -8 * (d.abs() + e) + 1e-37).all()
    assert ((db.double() - d.sum(0)).abs() <= e.sum(0) + (T + 20) * U * (d.abs() + e).sum(0)).all()
    d = dz.double()
    want = d @ w.double().t().contiguous()
    tol = (N + 8) * U * (d.abs() @ w.double().abs().t().contiguous())
    assert ((dx.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-37).all()
    xt = x.double().t().contiguous()
    assert ((dw.double() - xt @ d).abs() <= (T + 8) * U * (xt.abs() @ d.abs())).all()
    # what is not wanted is left out, and the rest keeps its bits; dz in dy's place
    some = _lib.moe_linear_backward(dy, x, w, act=act, z=z, want_dw=False, want_db=False)
    assert torch.equal(some[1], dx) and some[2] is None and some[3] is None
    some = _lib.moe_linear_backward(dy, x, w, act=act, z=z, want_dx=False)
    assert some[1] is None and torch.equal(some[2], dw) and torch.equal(some[3], db)
    here = dy.clone()
    some = _lib.moe_linear_backward(here, x, w, act=act, z=z, dz=here)
    assert some[0] is here and torch.equal(here, dz) and torch.equal(some[1], dx) and torch.equal(some[2], dw)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """dz against central differences of the activation in 64 bits: h = 10^-5 leaves h^2 of the third derivative and
    10^-11 of rounding; dz itself is a bf16."""
    z = torch.linspace(-12, 12, 64 * 64, device="cuda").view(64, 64).to(BF)
    dy = torch.ones_like(z)
    dz = _lib.moe_linear_backward(dy, rand(1, 64, 64, dtype=BF), rand(2, 64, 64, dtype=BF), act=act, z=z)[0]
    v, h = z.double(), 1e-5
    diff = (act64(act, v + h) - act64(act, v - h)) / (2 * h)
    assert ((dz.double() - diff).abs() <= 2.0 ** -8 * diff.abs() + 2.0 ** -18 * (1 + v.abs())).all()


@pytest.mark.parametrize("act", ACTS)
def test_far_values_of_the_activations(act):
    """Far from 0 the activations are 0 or z, and their slopes 0 or 1, without a NaN; a NaN stays one."""
    T = 4
    x = torch.zeros((T, 64), dtype=BF, device="cuda")
    bias = torch.tensor([-3e38, -1e30, -1e4, -200.0, -100.0, 100.0, 1e4, 1e30] * 8, device="cuda")
    y, z = _lib.moe_linear(x, torch.zeros((64, 64), dtype=BF, device="cuda"), bias=bias, act=act, want_z=True)
    want = bias if act == "none" else bias.clamp(min=0)
    assert torch.equal(y, want.to(BF).expand(T, 64)) and torch.equal(z, bias.to(BF).expand(T, 64))
    dz = _lib.moe_linear_backward(torch.ones_like(y), x, x[:1].expand(64, 64).contiguous(), act=act, z=z)[0]
    assert torch.equal(dz.float(), torch.ones_like(bias).expand(T, 64) if act == "none" else (bias > 0).float().expand(T, 64))
    bias[5] = float("nan")
    y, _ = _lib.moe_linear(x, torch.zeros((64, 64), dtype=BF, device="cuda"), bias=bias, act=act)
    assert torch.isnan(y[:, 5]).all() and int(torch.isnan(y).sum()) == T


@pytest.mark.parametrize("T", [3, 80, 5000])
def test_rows_do_not_mix(T):
    """A NaN and an infinity in one row of x reach that row only, in every form."""
    x, w = rand(1, T, 256, dtype=BF), rand(2, 256, 704, dtype=BF)
    y = _lib.moe_linear(x, w)[0]
    x[1, 3], x[T - 1, 9] = float("nan"), float("inf")
    got = _lib.moe_linear(x, w)[0]
    rows = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(got[rows], y[rows]) and torch.isnan(got[1]).all() and not torch.isfinite(got[T - 1]).any()


def test_no_tokens():
    x, w = torch.empty((0, 128), dtype=BF, device="cuda"), rand(2, 128, 192, dtype=BF)
    y, z = _lib.moe_linear(x, w, act="gelu", want_z=True)
    assert y.shape == z.shape == (0, 192)
    dw, db = torch.full((128, 192), 5.0, device="cuda"), torch.full((192,), 5.0, device="cuda")
    dz, dx, _, _ = _lib.moe_linear_backward(y, x, w, act="gelu", z=z, dw=dw, db=db)
    assert dz.shape == (0, 192) and dx.shape == (0, 128) and (dw == 0).all() and (db == 0).all()


def test_outputs_past_2_31_values():
    """Whole numbers again, 2^31 outputs and more: rows at both ends and around the border, bit for bit."""
    T, Kd, N = 520001, 64, 4160
    x, w, dy1 = ints(1, T, Kd), ints(2, Kd, N), ints(3, N, top=1)
    res = torch.zeros((T, N), dtype=BF, device="cuda")
    border = (1 << 31) // N
    probe = torch.tensor([0, 1, 255, 256, border - 1, border, border + 1, T - 2, T - 1], device="cuda")
    res[probe] = ints(4, len(probe), N, top=60)
    print(f"[linear] {T} x {Kd} x {N}", flush=True)
    y, z = _lib.moe_linear(x, w, act="relu", residual=res, want_z=True)
    want = x[probe].double() @ w.double()
    assert torch.equal(z[probe], want.float().to(BF))
    assert torch.equal(y[probe], (want.clamp(min=0) + res[probe].double()).float().to(BF))
    del res
    dy = y.copy_(dy1)  # the same gradient in every row
    dz, dx, dw, db = _lib.moe_linear_backward(dy, x, w, act="relu", z=z, dz=dy)
    d = dy1.double() * (want > 0)
    assert torch.equal(dz[probe], d.to(BF))
    assert torch.equal(dx[probe], (d @ w.double().t().contiguous()).float().to(BF))
    sign = torch.zeros(N, dtype=torch.float64, device="cuda")
    grad = torch.zeros((Kd, N), dtype=torch.float64, device="cuda")
    for lo in range(0, T, 40000):
        part = dy1.double() * (x[lo:lo + 40000].double() @ w.double() > 0)
        sign += part.sum(0)
        grad += x[lo:lo + 40000].double().t().contiguous() @ part
    assert torch.equal(db.double(), sign) and torch.equal(dw.double(), grad)


def test_workspace_of_the_caller_and_what_is_behind_it():
    x, w, dy = rand(1, 70, 1024, dtype=BF), rand(2, 1024, 128, dtype=BF), rand(3, 70, 128, dtype=BF)
    n = _lib.moe_linear_workspace_size(70, 1024, 128)
    m = _lib.moe_linear_backward_workspace_size(70, 1024, 128)
    assert n > 0 and m > 0
    ws = torch.full((max(n, m) + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    assert torch.equal(_lib.moe_linear(x, w, ws=ws[:n])[0], _lib.moe_linear(x, w)[0])
    assert (ws[n:] == 0xA5).all()
    ws.fill_(0xA5)
    got, want = _lib.moe_linear_backward(dy, x, w, ws=ws[:m]), _lib.moe_linear_backward(dy, x, w)
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3]) and (ws[m:] == 0xA5).all()


def test_refusals():
    x, w, b = rand(1, 4, 128, dtype=BF), rand(2, 128, 64, dtype=BF), rand(3, 64)
    y = rand(4, 4, 64, dtype=BF)
    for kw in (dict(act="tanh"), dict(bias=b.to(BF)), dict(bias=b[:32].contiguous()), dict(residual=x), dict(z=y.float()),
               dict(y=x), dict(w=w.t()), dict(w=w[:64].contiguous()), dict(x=x.float()), dict(x=x[0]), dict(ws=b)):
        with pytest.raises(_lib.MoeError):
            _lib.moe_linear(**dict(dict(x=x, w=w), **kw))
    with pytest.raises(_lib.MoeError):
        _lib.moe_linear(rand(5, 4, 96, dtype=BF), rand(6, 96, 64, dtype=BF))
    for kw in (dict(act="gelu"), dict(act="gelu", z=x), dict(dz=x), dict(dw=w), dict(dx=y), dict(db=b.double()),
               dict(dy=x), dict(act="gelu", z=y, dz=x)):
        with pytest.raises(_lib.MoeError):
            _lib.moe_linear_backward(**dict(dict(dy=y, x=x, w=w), **kw))
