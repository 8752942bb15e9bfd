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
