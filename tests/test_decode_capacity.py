"""The row capacity of a decode step on a share of the experts: no pair is dropped."""
import numpy as np
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, pipeline, synth

SHARE = synth.WORKLOADS["ep_share_4k"].scaled(H=128, F=192)  # 32 of 256 experts, top 8


@pytest.mark.parametrize("T", [1, 2, 37, 512])
@pytest.mark.parametrize("EL", [4, 32, 256])
def test_capacity_holds_every_pair_that_can_be_local(T, EL):
    shape = SHARE.scaled(T=T, e_local=EL)
    buf = pipeline.MoeBuffers.allocate(shape, weights4=True, device="cpu")
    assert buf.cap == T * min(8, EL) and buf.h.shape[0] == buf.src.numel() == buf.cap
    assert buf.ws4.numel() >= _lib.moe_gemm4_combine_workspace_size(buf.cap, shape.H)
    assert pipeline.MoeBuffers.allocate(shape, cap=3, weights4=True, device="cpu").cap == 3
    # the other forms keep the shape's own capacity
    assert pipeline.MoeBuffers.allocate(shape, device="cpu", backward=False).cap == shape.cap


@pytest.mark.gpu
@pytest.mark.parametrize("T,seed,local", [(1, 10, 3), (2, 35, 6), (4, 77, 9), (5, None, 40)])
def test_decode_step_with_more_rows_than_twice_the_expected(T, seed, local):
    """Routings that exceed the shape's own capacity (the last: every token on the share's first experts): every
    local pair has its row, and the output is the gated sum of all of them."""
    shape = SHARE.scaled(T=T)
    inp = synth.make_inputs(shape, seed=seed or 0)
    if seed is None:
        inp["logits"][:, :8] += 100.0
    assert local > shape.cap
    dev = pipeline.to_device(inp)
    dev.update(pipeline.pack_weights4(dev))
    buf = pipeline.MoeBuffers.allocate(shape, weights4=True)
    out = pipeline.forward4(buf, dev)
    idx, pos = buf.topk_idx.cpu(), buf.pos.cpu()
    assert int(buf.status[0]) == 0 and int(buf.offsets[-1]) == local
    assert torch.equal(pos >= 0, idx < 32) and int((pos >= 0).sum()) == local
    # from the packed values: h rounds to bf16 as the call's does, the rest in float64
    w = {k: _lib.moe_unpack4(*dev[k + "4"], kd).double() for k, kd in (("w_gate", 128), ("w_up", 128), ("w_down", 192))}
    x = dev["x"].double()
    for t in range(T):
        want, mag = torch.zeros(128, dtype=torch.float64, device="cuda"), 0.0
        for k in np.flatnonzero(pos[t].numpy() >= 0):
            e, g = int(idx[t, k]), float(buf.gates[t, k])
            h = buf.h[int(pos[t, k])].double()
            a, b = x[t] @ w["w_gate"][e], x[t] @ w["w_up"][e]
            # fp32 sums of 128 products, the sigmoid and one rounding to bf16
            ea, eb = (128 * 2.0 ** -24 * (x[t].abs() @ w[m][e].abs()) for m in ("w_gate", "w_up"))
            s = torch.sigmoid(a)
            tol = 1.1 * ea * b.abs() + (a * s).abs() * eb + 1.1 * ea * eb + (2.0 ** -8 + 2.0 ** -18) * (a * s * b).abs()
            assert ((h - a * s * b).abs() <= tol + 1e-37).all()
            want += g * (h @ w["w_down"][e])
            mag += g * (h.abs() @ w["w_down"][e].abs())
        # fp32 sums of 192 products and of 8 gated rows, and one rounding to bf16
        assert ((out[t].double() - want).abs() <= (192 + 16) * 2.0 ** -24 * mag + 2.0 ** -8 * want.abs() + 1e-37).all()


def test_4bit_buffers_refuse_a_backward():
    """An explicit backward or checkpoint was dropped without a word; a shape that has a backward may still serve."""
    for kw in (dict(backward=True), dict(checkpoint8=True), dict(backward=True, checkpoint8=True)):
        with pytest.raises(_lib.MoeError):
            pipeline.MoeBuffers.allocate(SHARE.scaled(T=4), weights4=True, device="cpu", **kw)
    for shape, backward in ((SHARE.scaled(T=4, backward=True), None), (SHARE.scaled(T=4), False)):
        buf = pipeline.MoeBuffers.allocate(shape, weights4=True, device="cpu", backward=backward)
        assert buf.dx is None and buf.ab8 is None and not buf.checkpoint8


def test_4bit_buffers_refuse_the_steps_of_the_other_forward():
    """There is no y and no backward in them."""
    buf = pipeline.MoeBuffers.allocate(SHARE.scaled(T=4), weights4=True, device="cpu")
    for call in (lambda: pipeline.expert_down(buf, None), lambda: pipeline.combine(buf),
                 lambda: pipeline.forward(buf, {}), lambda: pipeline.backward(buf, {})):
        with pytest.raises(_lib.MoeError):
            call()
    with pytest.raises(_lib.MoeError):
        pipeline.backward(pipeline.MoeBuffers.allocate(SHARE.scaled(T=4), device="cpu", backward=False), {})
