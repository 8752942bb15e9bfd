"""Layers that share h: the 8-bit checkpoint keeps nothing in it between forward and backward."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, pipeline, synth

SHAPE = synth.WORKLOADS["ep_share_4k"].scaled(T=512, H=256, F=192, backward=True)


def test_allocate_takes_a_shared_h():
    allocate = pipeline.MoeBuffers.allocate
    h = torch.empty((SHAPE.cap + 5, SHAPE.F), dtype=torch.bfloat16)
    layers = [allocate(SHAPE, device="cpu", checkpoint8=True, h=h) for _ in range(2)]
    assert layers[0].h is h and layers[1].h is h
    assert allocate(SHAPE, device="cpu", backward=False, h=h).h is h
    assert allocate(SHAPE, device="cpu", weights4=True, cap=SHAPE.cap, h=h).h is h
    # what a layer keeps of a row for the backward: q8 and scales of a and b
    kept = sum(t.element_size() * t.shape[1] for t in (layers[0].ab8, layers[0].ab8_scale))
    assert kept == 2 * SHAPE.F * 33 // 32 and layers[0].ab is None
    for kw in (dict(h=h),                                                      # h is saved for the backward
               dict(checkpoint8=True, h=h[:SHAPE.cap - 1]),
               dict(checkpoint8=True, h=h.float()),
               dict(checkpoint8=True, h=h[:, :128].contiguous()),
               dict(checkpoint8=True, h=h[:, :128]),
               dict(checkpoint8=True, h=torch.empty_like(h, device="meta"))):
        with pytest.raises(_lib.MoeError):
            allocate(SHAPE, device="cpu", **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("zero_copy", [False, True])
def test_two_layers_share_h(zero_copy):
    """Forward, forward, backward, backward through one h: the bits of layers with an h of their own."""
    dev = [pipeline.to_device(synth.make_inputs(SHAPE, seed=70 + i, d_out=True)) for i in range(2)]
    own = [pipeline.MoeBuffers.allocate(SHAPE, checkpoint8=True, zero_copy=zero_copy) for _ in dev]
    h = torch.full_like(own[0].h, float("nan"))
    shared = [pipeline.MoeBuffers.allocate(SHAPE, checkpoint8=True, zero_copy=zero_copy, h=h) for _ in dev]
    for layers in (own, shared):
        for buf, inp in zip(layers, dev):
            pipeline.forward(buf, inp)
        for buf, inp in reversed(list(zip(layers, dev))):
            pipeline.backward(buf, inp)
    assert int(own[0].offsets[-1]) != int(own[1].offsets[-1])
    for a, b in zip(own, shared):
        for n in ("out", "dx", "dw_gate", "dw_up", "dw_down", "dlogits"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n
