"""The whole layer for a few tokens (moe_layer_few) against its formula in 64 bits and against the layer's own steps."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, pipeline, synth

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def normal(seed, *shape, std=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(BF)


def layer(seed, T, H, F, E, EL, std=0.05):
    logits = normal(seed, T, E).float() + normal(seed + 1, T, E, std=0.01).float()
    return logits, normal(seed + 2, T, H), normal(seed + 3, EL, H, F, std=std), normal(seed + 4, EL, H, F, std=std), \
        normal(seed + 5, EL, F, H, std=std)


def reference(logits, x, K, e0, wg, wu, wd, residual):
    """(choices, gates, out in float64, its tolerance): fp32 sums of H and F products, h rounded to bf16 (2^-8), the
    exponentials and quotients of the gates and of the sigmoid within 2^-18, a sum of K gated rows, one rounding."""
    T, EL, H, F = x.shape[0], wg.shape[0], wg.shape[1], wg.shape[2]
    rows = logits.double().cpu()
    idx = torch.tensor([sorted(range(len(r)), key=lambda e: (-r[e], e))[:K] for r in rows.tolist()], dtype=torch.int64)
    gates = torch.softmax(rows.gather(1, idx), 1)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    if residual is not None:
        out += residual
    tol += 2.0 ** -24 * out.abs()
    for j in range(EL):
        pairs = [(t, k) for t in range(T) for k in range(K) if idx[t, k] == e0 + j]
        if not pairs:
            continue
        at = torch.tensor([t for t, _ in pairs], device="cuda")
        g = torch.tensor([float(gates[p]) for p in pairs], dtype=torch.float64, device="cuda")[:, None]
        xr, g_w, u_w, d_w = x[at].double(), wg[j].double(), wu[j].double(), wd[j].double()
        a, b = xr @ g_w, xr @ u_w
        ea, eb = (H * 2.0 ** -24 * (xr.abs() @ w.abs()) for w in (g_w, u_w))
        s = a * torch.sigmoid(a)
        h = s * b
        eh = 1.1 * ea * b.abs() + s.abs() * eb + 1.1 * ea * eb + (2.0 ** -8 + 2.0 ** -18) * h.abs()
        y = h @ d_w
        ey = eh @ d_w.abs() + F * 2.0 ** -24 * ((h.abs() + eh) @ d_w.abs())
        out[at] += g * y
        tol[at] += g * (ey + (2.0 ** -18 + (K + 2) * 2.0 ** -24) * (y.abs() + ey))
    return idx.to(torch.int32), gates, out, tol + 2.0 ** -8 * (out.abs() + tol) + 1e-37


CASES = [
    # T, H, F, E, e0, EL, K
    (1, 64, 64, 1, 0, 1, 1),
    (1, 128, 256, 8, 0, 8, 2),
    (2, 192, 64, 65, 0, 65, 3),
    (3, 192, 128, 7, 2, 3, 4),
    (15, 320, 192, 130, 60, 70, 8),
    (16, 256, 64, 16, 0, 16, 16),
    (17, 128, 320, 3, 0, 3, 3),
    (31, 704, 192, 300, 299, 1, 6),
    (33, 2048, 768, 128, 0, 128, 8),
    (48, 64, 64, 8, 0, 2, 8),
    (64, 192, 128, 512, 100, 200, 16),
    (64, 448, 576, 9, 0, 9, 9),
    (64, 64, 64, 512, 0, 512, 16),
    (20, 128, 1088, 2, 1, 1, 2),
]


@pytest.mark.parametrize("T,H,F,E,e0,EL,K", CASES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_against_the_formula(T, H, F, E, e0, EL, K, with_residual):
    logits, x, wg, wu, wd = layer(T + H, T, H, F, E, EL)
    residual = normal(99, T, H) if with_residual else None
    idx, gates, want, tol = reference(logits, x, K, e0, wg, wu, wd, residual)
    print(f"[few] T={T} H={H} F={F} E={E} share {e0}+{EL} K={K}", flush=True)
    out, got_idx, got_gates = _lib.moe_layer_few(logits, x, K, e0, wg, wu, wd, residual=residual)
    assert torch.equal(got_idx.cpu(), idx)
    assert ((got_gates.double().cpu() - gates).abs() <= 2.0 ** -18 * gates).all()
    err = (out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    # the choices and gates of the layer's own routing, bit for bit, and the same bits again
    r_idx, r_gates = _lib.moe_route(logits, K)
    assert torch.equal(got_idx, r_idx) and torch.equal(got_gates, r_gates)
    again = _lib.moe_layer_few(logits, x, K, e0, wg, wu, wd, residual=residual)[0]
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("T", [1, 20, 64])
def test_every_token_on_the_same_experts(T):
    """64 rows on each of K experts, and none on the others."""
    logits, x, wg, wu, wd = layer(5, T, 256, 192, 16, 16)
    logits[:, 3] += 50
    logits[:, 15] += 40
    idx, _, want, tol = reference(logits, x, 2, 0, wg, wu, wd, None)
    assert (idx[:, 0] == 3).all() and (idx[:, 1] == 15).all()
    out, got_idx, _ = _lib.moe_layer_few(logits, x, 2, 0, wg, wu, wd)
    assert torch.equal(got_idx.cpu(), idx)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("EL", [0, 2])
@pytest.mark.parametrize("with_residual", [False, True])
def test_tokens_without_a_local_expert(EL, with_residual):
    """No pair is local (or there is no local expert at all): the residual as it is, or zeros; and where one token of
    several has one, the others' rows."""
    T, H = 5, 192
    logits, x, wg, wu, wd = layer(8, T, H, 64, 6, EL)
    logits[:, 4:] -= 100
    residual = normal(9, T, H) if with_residual else None
    empty = residual if with_residual else torch.zeros((T, H), dtype=BF, device="cuda")
    out, _, _ = _lib.moe_layer_few(logits, x, 3, 4 if EL else 6, wg, wu, wd, residual=residual)
    assert torch.equal(out, empty)
    if EL:
        logits[2, 5] += 300
        out, idx, _ = _lib.moe_layer_few(logits, x, 3, 4, wg, wu, wd, residual=residual)
        assert int(idx[2, 0]) == 5
        rest = [0, 1, 3, 4]
        assert torch.equal(out[rest], empty[rest])
        _, _, want, tol = reference(logits, x, 3, 4, wg, wu, wd, residual)
        assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("H,F,E,K", [(256, 256, 128, 8), (320, 192, 16, 4), (128, 128, 8, 8), (192, 2048, 64, 2)])
def test_bits_in_every_form(H, F, E, K):
    """A token alone, and among as many others as each form of the kernels takes: the same bits."""
    logits, x, wg, wu, wd = layer(23, 64, H, F, E, E)
    out = _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd)[0]
    for T in (1, 2, 5, 15, 16, 17, 31, 32, 33, 48, 63):
        print(f"[few] forms T={T} H={H} F={F} E={E} K={K}", flush=True)
        got = _lib.moe_layer_few(logits[:T].contiguous(), x[:T].contiguous(), K, 0, wg, wu, wd)[0]
        assert torch.equal(got, out[:T])


def test_large_values_between_the_products():
    """h past the largest bf16 is an infinity there, as one rounding makes it, and no NaN."""
    T, H, F = 3, 64, 64
    logits = torch.zeros((T, 1), device="cuda")
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[:, 0] = 1
    wg, wu = (torch.zeros((1, H, F), dtype=BF, device="cuda") for _ in range(2))
    wd = torch.zeros((1, F, H), dtype=BF, device="cuda")
    wg[:, 0], wu[:, 0, :] = 2.0 ** 64, 2.0 ** 62  # silu(2^64) * 2^62 = 2^126
    wd[0, 0] = 1.0
    out = _lib.moe_layer_few(logits, x, 1, 0, wg, wu, wd)[0]
    assert torch.equal(out, torch.full_like(out, 2.0 ** 126))
    wu[:, 0, :] = 2.0 ** 64
    wd[:] = 1.0
    out = _lib.moe_layer_few(logits, x, 1, 0, wg, wu, wd)[0]
    assert torch.isinf(out).all() and (out > 0).all()


def test_ties_go_to_the_lowest_expert():
    T, E, K = 9, 200, 5
    logits, x, wg, wu, wd = layer(11, T, 64, 64, E, E)
    logits = logits.round()  # many equal scores, -0 among them
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    logits[1, 1::2] = 0.0
    idx = _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd)[1].cpu()
    for t, row in enumerate(logits.cpu().tolist()):
        assert idx[t].tolist() == sorted(range(E), key=lambda e: (-row[e], e))[:K]


def test_scores_of_minus_infinity_and_nan():
    """A router that masks experts gives them -inf: more choices than experts are left get a gate of 0, and a token with
    none left, or with a NaN, gates that are NaN, as the layer's routing says; the other tokens are as they were."""
    T, K = 12, 4
    logits, x, wg, wu, wd = layer(12, T, 128, 64, 70, 70)
    inf = float("inf")
    logits[1, 2:] = -inf  # two experts left of four wanted
    logits[2] = -inf
    logits[3, 5] = float("nan")
    logits[4, 7] = inf
    out, idx, gates = _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd)
    r_idx, r_gates = _lib.moe_route(logits, K)
    rows = [t for t in range(T) if t != 3]  # where a NaN is ranked is not said
    assert torch.equal(idx[rows], r_idx[rows])
    assert torch.equal(gates[rows].view(torch.int32), r_gates[rows].view(torch.int32))
    assert idx[1].tolist()[2:] == [2, 3] and (gates[1, 2:] == 0).all() and torch.isnan(gates[2]).all()
    assert ((idx >= 0) & (idx < 70)).all()
    fine = [0, 1] + list(range(5, T))
    clean = logits.clone()
    clean[2:5] = 0.0
    assert torch.equal(out[fine], _lib.moe_layer_few(clean, x, K, 0, wg, wu, wd)[0][fine])
    assert torch.isfinite(out[fine]).all()


def test_a_token_does_not_change_with_the_others():
    """NaN, infinities and other routes in the other tokens leave a token's bits as they are, and so does their number."""
    T, K = 40, 4
    logits, x, wg, wu, wd = layer(13, T, 256, 128, 12, 12)
    out = _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd)[0]
    other, xo = logits.clone(), x.clone()
    keep = [0, 7, 39]
    change = [t for t in range(T) if t not in keep]
    other[change] = other[change].flip(1)
    xo[change[::2]] = float("nan")
    xo[change[1::2]] = float("inf")
    assert torch.equal(_lib.moe_layer_few(other, xo, K, 0, wg, wu, wd)[0][keep], out[keep])
    assert torch.equal(_lib.moe_layer_few(logits[:7].contiguous(), x[:7].contiguous(), K, 0, wg, wu, wd)[0], out[:7])
    assert torch.equal(_lib.moe_layer_few(logits[7:8].contiguous(), x[7:8].contiguous(), K, 0, wg, wu, wd)[0], out[7:8])


def test_a_nan_in_an_expert_reaches_its_tokens_only():
    logits, x, wg, wu, wd = layer(17, 6, 128, 64, 8, 8)
    wd[3, 5, 70] = float("nan")
    out, idx, _ = _lib.moe_layer_few(logits, x, 2, 0, wg, wu, wd)
    hit = (idx == 3).any(1)
    bad = torch.isnan(out)
    assert hit.any() and not hit.all()
    assert bad[hit][:, 70].all() and int(bad.sum()) == int(hit.sum())


def test_residual_in_place_and_buffers_given():
    logits, x, wg, wu, wd = layer(19, 21, 320, 64, 10, 10)
    residual = normal(20, 21, 320)
    want, idx, gates = _lib.moe_layer_few(logits, x, 3, 0, wg, wu, wd, residual=residual)
    need = _lib.moe_layer_few_workspace_size(21, 3, 10, 320, 64)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    stream = residual.clone()
    got = _lib.moe_layer_few(logits, x, 3, 0, wg, wu, wd, residual=stream, out=stream, ws=ws,
                             topk_idx=torch.empty_like(idx), gates=torch.empty_like(gates))
    assert got[0] is stream and torch.equal(stream, want) and torch.equal(got[1], idx) and torch.equal(got[2], gates)
    assert (ws[need:] == 0xA5).all()
    # the tokens' rows themselves
    want = _lib.moe_layer_few(logits, x, 3, 0, wg, wu, wd, residual=x.clone())[0]
    assert torch.equal(_lib.moe_layer_few(logits, x, 3, 0, wg, wu, wd, residual=x, out=x, ws=ws)[0], want)


def test_no_tokens():
    _, _, wg, wu, wd = layer(23, 1, 64, 64, 4, 4)
    out, idx, gates = _lib.moe_layer_few(torch.empty((0, 4), device="cuda"), torch.empty((0, 64), dtype=BF, device="cuda"),
                                         2, 0, wg, wu, wd)
    assert out.shape == (0, 64) and idx.shape == gates.shape == (0, 2)


@pytest.mark.parametrize("T", [1, 37, 64])
def test_pipeline_form_matches_the_layers_steps(T):
    """forward_few against forward on the same inputs: both round h to bf16; the steps round the experts' rows as well."""
    shape = synth.WORKLOADS["tiny"].scaled(T=T)
    dev = pipeline.to_device(synth.make_inputs(shape, seed=3))
    few = pipeline.FewBuffers.allocate(shape)
    out = pipeline.forward_few(few, dev).clone()
    buf = pipeline.MoeBuffers.allocate(shape, backward=False)
    pipeline.forward(buf, dev)
    assert torch.equal(few.topk_idx, buf.topk_idx) and torch.equal(few.gates, buf.gates)
    _, _, want, tol = reference(dev["logits"], dev["x"], shape.K, 0, dev["w_gate"], dev["w_up"], dev["w_down"], None)
    assert ((out.double() - want).abs() <= tol).all()
    rows = 2.0 ** -8 * torch.stack([(buf.gates[t, :, None] * buf.y[buf.pos[t].long()].abs()).sum(0) for t in range(T)])
    assert ((buf.out.double() - want).abs() <= tol + rows).all()


def test_two_streams_with_a_workspace_each():
    args = [layer(30 + i, 30 + i, 512, 256, 32, 32) for i in range(2)]
    want = [_lib.moe_layer_few(a[0], a[1], 4, 0, *a[2:])[0] for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = []
    for _ in range(3):
        got.append([_lib.moe_layer_few(a[0], a[1], 4, 0, *a[2:], stream=s)[0] for a, s in zip(args, streams)])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    T, K = 24, 3
    logits, x, wg, wu, wd = layer(40, T, 384, 192, 24, 24)
    ws = torch.empty(_lib.moe_layer_few_workspace_size(T, K, 24, 384, 192), dtype=torch.uint8, device="cuda")
    out, idx, gates = _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.moe_layer_few(logits, x, K, 0, wg, wu, wd, ws=ws, out=out, topk_idx=idx, gates=gates)
    for seed in (41, 45, 49):
        l2, x2 = layer(seed, T, 384, 192, 24, 24)[:2]
        want = _lib.moe_layer_few(l2, x2, K, 0, wg, wu, wd)
        logits.copy_(l2)
        x.copy_(x2)
        ws.fill_(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, idx, gates), want):
            assert torch.equal(a, b)


def test_refusals():
    logits, x, wg, wu, wd = layer(50, 4, 128, 64, 8, 8)
    bad = [
        dict(x=x[:, :64].contiguous()), dict(x=x.float()), dict(x=x.t()), dict(w_down=wd[:4].contiguous()),
        dict(w_up=wu.transpose(1, 2)), dict(logits=logits.double()), dict(residual=x[:2].contiguous()),
        dict(out=torch.empty((5, 128), dtype=BF, device="cuda")), dict(K=0), dict(K=9), dict(e_begin=1), dict(e_begin=-1),
        dict(gates=torch.empty((4, 2), dtype=torch.float64, device="cuda")), dict(ws=torch.empty(8, device="cuda")),
    ]
    for kw in bad:
        args = dict(dict(logits=logits, x=x, K=2, e_begin=0, w_gate=wg, w_up=wu, w_down=wd), **kw)
        with pytest.raises(_lib.MoeError):
            _lib.moe_layer_few(**args)
    with pytest.raises(_lib.MoeError):
        _lib.moe_layer_few(normal(1, 65, 8).float(), normal(2, 65, 128), 2, 0, wg, wu, wd)
