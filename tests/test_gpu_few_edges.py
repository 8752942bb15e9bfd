"""The few-token layer's h in two bf16 values: what the second holds, and infinite weights against it."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib
from test_gpu_few import BF, layer

pytestmark = pytest.mark.gpu

# T, experts, K: a pass of 16 rows of an expert, passes of 32 and of 64, several passes, and rows that fill none
FORMS = [(1, 6, 2), (20, 6, 2), (24, 2, 2), (64, 3, 2), (64, 1, 1), (48, 2, 2)]


def silu_up(x, wg, wu):
    a = x.double() @ wg.double()
    return a * torch.sigmoid(a) * (x.double() @ wu.double())


@pytest.mark.parametrize("T,E,K", FORMS)
def test_infinite_weights_of_the_down_product(T, E, K):
    """h . w_down with an infinite weight is an infinity of h's sign (no h is 0), and a NaN only where infinities of both
    signs meet; the other columns keep their bits, and so do the tokens without that expert."""
    H, F = 192, 128
    logits, x, wg, wu, wd = layer(61 + T, T, H, F, E, E)
    inf = float("inf")
    clean, idx, gates = _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd)
    j, bad = int(idx[0, 0]), wd.clone()
    bad[j, 5, 70], bad[j, 77, 71], bad[j, 127, 191] = inf, -inf, inf
    bad[j, 3, 0], bad[j, 90, 0] = inf, -inf
    print(f"[few] infinite weights T={T} E={E} K={K}", flush=True)
    out = _lib.moe_layer_few(logits, x, K, 0, wg, wu, bad)[0].double()
    h = silu_up(x, wg[j], wu[j])
    hit = (idx == j).any(1)
    assert (h[hit] != 0).all() and (gates[idx == j] > 0).all()
    want = clean.double()
    for n in (0, 70, 71, 191):
        w = torch.where(torch.isinf(bad[j, :, n]), bad[j, :, n].double(), 0.0)
        at = torch.nonzero(torch.isinf(w)).reshape(-1)
        terms = h[hit][:, at].sign() * w[at]
        want[hit, n] = terms.sum(1)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out, nan=0.0, posinf=inf, neginf=-inf),
                       torch.nan_to_num(want, nan=0.0, posinf=inf, neginf=-inf))


def test_infinite_weights_and_an_h_that_one_value_holds():
    """h = 2^126 exactly: the rest is 0, which times an infinity would be a NaN."""
    T, H, F = 3, 64, 64
    logits = torch.zeros((T, 1), device="cuda")
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[:, 0] = 1
    wg, wu = (torch.zeros((1, H, F), dtype=BF, device="cuda") for _ in range(2))
    wg[:, 0], wu[:, 0, :] = 2.0 ** 64, 2.0 ** 62
    wd = torch.zeros((1, F, H), dtype=BF, device="cuda")
    wd[0, 4, :32] = float("inf")
    out = _lib.moe_layer_few(logits, x, 1, 0, wg, wu, wd)[0]
    assert torch.isposinf(out[:, :32]).all() and (out[:, 32:] == 0).all()


def rows_of(h, gates, idx, wd):
    """Gated sums of the experts' rows from h [E, T, F], and of their magnitudes."""
    out, mag = (torch.zeros(h.shape[1], wd.shape[2], dtype=torch.float64, device="cuda") for _ in range(2))
    for j in range(wd.shape[0]):
        g = (gates * (idx == j)).sum(1, keepdim=True)
        out += g * (h[j] @ wd[j].double())
        mag += g * (h[j].abs() @ wd[j].double().abs())
    return out, mag


@pytest.mark.parametrize("T,E,K", FORMS)
@pytest.mark.parametrize("H,F", [(64, 128), (192, 320)])
def test_h_keeps_sixteen_bits(T, E, K, H, F):
    """Every token has one 1, so that gate and up are single weights, without a sum's roundings: h is off by its sigmoid
    (2^-18), a product and the rounding of its second value (2^-8 of 2^-8); the down product's fp32 sums of 2F products and
    of K gated rows add theirs, the output rounds once.  An h that is rounded to one bf16 fails the same tolerance, by the
    outputs that cancel."""
    logits, _, wg, wu, wd = layer(81 + T, T, H, F, E, E, std=1.0)
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[torch.arange(T), torch.arange(T) * 7 % H] = 1.0
    print(f"[few] two values T={T} E={E} K={K} H={H} F={F}", flush=True)
    out, idx, gates = _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd)
    g64 = torch.softmax(logits.double().gather(1, idx.long()), 1)
    h = torch.stack([silu_up(x, wg[j], wu[j]) for j in range(E)])
    want, mag = rows_of(h, g64, idx, wd)
    tol = (2.0 ** -16 + 2 * 2.0 ** -18 + (2 * F + K + 4) * 2.0 ** -24) * mag
    tol = tol + 2.0 ** -8 * (want.abs() + tol) + 1e-37
    err = (out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    once = rows_of(h.to(BF).double(), g64, idx, wd)[0]
    assert ((once - want).abs() > tol).any()  # what the tolerance would not let pass
