"""A block's feed-forward half (block.py): norm, router, experts and shared expert together, against 64 bits."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, block, synth

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(seed, *shape, std=1.0, shift=0.0, dtype=BF):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std + shift).to(dtype)


def weights(shape, shared, rms, seed=0):
    H, F, E, EL = shape.H, shape.F, shape.E, shape.EL
    p = {"norm_weight": rand(seed + 1, H, std=0.2, shift=1.0, dtype=torch.float32),
         "w_r": rand(seed + 2, H, E, std=0.1), "router_bias": rand(seed + 3, E, dtype=torch.float32),
         "w_gate": rand(seed + 4, EL, H, F, std=0.06), "w_up": rand(seed + 5, EL, H, F, std=0.06),
         "w_down": rand(seed + 6, EL, F, H, std=0.06)}
    if not rms:
        p["norm_bias"] = rand(seed + 7, H, std=0.2, dtype=torch.float32)
    if shared:
        p.update(shared_gate=rand(seed + 8, 1, H, shared, std=0.06), shared_up=rand(seed + 9, 1, H, shared, std=0.06),
                 shared_down=rand(seed + 10, 1, shared, H, std=0.06))
    return p


def reference(p, x, add, idx, e0, eps=1e-5):
    """s and out in 64 bits, the choice of experts taken from the call (a near tie may go either way)."""
    s = x if add is None else x + add
    mean = s.mean(1, keepdim=True) if "norm_bias" in p else torch.zeros_like(s[:, :1])
    y = (s - mean) / ((s - mean).square().mean(1, keepdim=True) + eps).sqrt() * p["norm_weight"]
    y = y + p.get("norm_bias", 0)
    logits = y @ p["w_r"] + p["router_bias"]
    gates = torch.softmax(logits.gather(1, idx), 1)
    silu = lambda a: a * torch.sigmoid(a)  # noqa: E731
    out = torch.zeros_like(y)
    for j in range(p["w_gate"].shape[0]):
        weight = (gates * (idx == e0 + j)).sum(1, keepdim=True)
        out = out + weight * ((silu(y @ p["w_gate"][j]) * (y @ p["w_up"][j])) @ p["w_down"][j])
    if "shared_down" in p:
        out = out + (silu(y @ p["shared_gate"][0]) * (y @ p["shared_up"][0])) @ p["shared_down"][0]
    return s, out


def near(name, got, want, roundings):
    """Normwise, so many roundings of at most 2^-8 in line."""
    rel = float((got.double() - want).norm() / want.norm())
    assert rel <= roundings * 2.0 ** -8, (name, rel)


SHAPE = synth.WORKLOADS["tiny"].scaled(H=192, F=128, E=64, K=3, backward=True)


@pytest.mark.parametrize("T,EL,shared,rms,f32", [(1, 64, 128, False, False), (37, 64, 64, True, False),
                                                 (300, 64, 0, False, True), (700, 24, 320, True, True)])
def test_training_step_against_autograd(T, EL, shared, rms, f32):
    shape = SHAPE.scaled(T=T, e_local=EL, e_begin=0 if EL == 64 else 8)
    dtype = torch.float32 if f32 else BF
    p = weights(shape, shared, rms)
    b = block.BlockBuffers.allocate(shape, shared=shared, x_dtype=dtype)
    x, add, d_out = rand(20, T, 192, std=1.5, shift=0.2, dtype=dtype), rand(21, T, 192), rand(22, T, 192)
    d_s = rand(23, T, 192, dtype=dtype)
    print(f"[block] T={T} EL={EL} shared={shared} rms={rms} f32={f32}", flush=True)
    s, out = block.forward(b, p, x, add)
    out = out.clone()
    g = block.backward(b, p, d_out, d_s)
    torch.cuda.synchronize()
    ref = {k: v.double().requires_grad_() for k, v in p.items()}
    x64 = x.double().requires_grad_()
    # the stored sum is the norm's input; its rounding passes the gradient on
    s64, out64 = reference(ref, x64 + (s.double() - x.double()), None, b.layer.topk_idx.long(), shape.e_begin)
    (out64 * d_out.double()).sum().add((s64 * d_s.double()).sum()).backward()
    assert torch.equal(s, (x.float() + add.float()).to(dtype))
    near("out", out, out64.detach(), 4)            # y, h, the experts' rows, out
    # dy_perm, (a, b), dab, dx_perm, dx, the sum of the parts, besides the forward's; the stream's gradient is added last
    near("x", g["x"], x64.grad, 10)
    for name in p:
        if name != "router_bias":
            near(name, g[name], ref[name].grad, 10)


@pytest.mark.parametrize("T", [1, 21, 64])
@pytest.mark.parametrize("shared", [0, 192])
def test_decode_step_against_the_training_form(T, shared):
    """Two blocks after each other, in the few-token form and in the other: both against 64 bits, and each other's
    choices."""
    shape = SHAPE.scaled(T=T, backward=False)
    x = rand(30, T, 192, std=1.5)
    runs = []
    for few in (True, False):
        s, add, got = x, None, []
        for i in range(2):
            p = weights(shape, shared, rms=True, seed=100 * i)
            b = block.BlockBuffers.allocate(shape, shared=shared, few=few)
            s_in, add_in = s, add
            s, add = block.forward(b, p, s, add)
            ref = {k: v.double() for k, v in p.items()}
            want_s, want = reference(ref, s.double(), None, b.layer.topk_idx.long(), 0)
            assert torch.equal(s, s_in if add_in is None else (s_in.float() + add_in.float()).to(BF))
            near("out", add, want, 4)
            got.append((b.layer.topk_idx.clone(), s, add))
        runs.append(got)
    assert torch.equal(runs[0][0][0], runs[1][0][0])  # the first block's scores are the same
    near("out", runs[0][0][2], runs[1][0][2].double(), 6)


def test_decode_block_captured_and_replayed():
    T, shared = 5, 64
    shape = SHAPE.scaled(T=T, backward=False)
    p = weights(shape, shared, rms=False)
    b, c = (block.BlockBuffers.allocate(shape, shared=shared, few=True) for _ in range(2))
    x, add = rand(40, T, 192), rand(41, T, 192)
    block.forward(b, p, x, add)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(b, p, x, add)
    for seed in (42, 44, 46):
        x.copy_(rand(seed, T, 192))
        add.copy_(rand(seed + 1, T, 192))
        want = block.forward(c, p, x, add)
        b.ws.fill_(seed)
        b.layer.ws.fill_(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.sum, want[0]) and torch.equal(b.out, want[1])


def test_training_step_captured_and_replayed():
    T, shared = 130, 64
    shape = SHAPE.scaled(T=T)
    p = weights(shape, shared, rms=False)
    b, c = (block.BlockBuffers.allocate(shape, shared=shared) for _ in range(2))
    x, add, d_out, d_s = (rand(50 + i, T, 192) for i in range(4))

    def step(buf):
        block.forward(buf, p, x, add)
        return block.backward(buf, p, d_out, d_s)

    step(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for seed in (60, 70, 80):
        for i, t in enumerate((x, add, d_out, d_s)):
            t.copy_(rand(seed + i, T, 192))
        want = step(c)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, c.out)
        for k in want:
            assert torch.equal(b.grads[k], want[k]), k


def test_refusals():
    with pytest.raises(_lib.MoeError):
        block.BlockBuffers.allocate(SHAPE.scaled(T=65), few=True)
    with pytest.raises(_lib.MoeError):
        block.BlockBuffers.allocate(SHAPE, few=True, backward=True)
    b = block.BlockBuffers.allocate(SHAPE.scaled(T=4))
    d = rand(1, 4, 192)
    with pytest.raises(_lib.MoeError):
        block.backward(b, weights(SHAPE, 0, True), d)
    b = block.BlockBuffers.allocate(SHAPE.scaled(T=4), backward=False)
    block.forward(b, weights(SHAPE, 0, True), d)
    with pytest.raises(_lib.MoeError):
        block.backward(b, weights(SHAPE, 0, True), d)
