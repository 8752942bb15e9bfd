"""moe_layer_few, moe_layer_norm and moe_linear and their backwards on the host: refusals before anything is enqueued,
workspace sizes, and the buffers that the binding makes for calls with stream=."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, pipeline, synth
from test_stream_argument_cpu import BF, F32, Traced, check, z

FAKE, MIS = 0x10000, 0x10002  # aligned and misaligned, never dereferenced
EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -4


def caller(name, **ok):
    fn = getattr(_lib.load(), name)
    return lambda **kw: fn(*dict(ok, **kw).values(), None)


def test_few_rejects():
    size = _lib.load().moe_layer_few_workspace_size
    need = size(16, 2, 8, 128, 64)
    call = caller("moe_layer_few", logits=FAKE, x=FAKE, T=16, E=8, K=2, e_begin=0, e_local=8, wg=FAKE, wu=FAKE, wd=FAKE,
                  H=128, F=64, res=None, idx=FAKE, gates=FAKE, out=FAKE, ws=FAKE, ws_bytes=need)
    for kw, want in ((dict(T=-1), EINVAL), (dict(T=65), EINVAL), (dict(E=513), EINVAL), (dict(K=0), EINVAL),
                     (dict(K=17, E=32), EINVAL), (dict(K=9), ESHAPE), (dict(H=96), ESHAPE), (dict(F=32), ESHAPE),
                     (dict(e_begin=1), EINVAL), (dict(e_begin=-1), EINVAL), (dict(e_begin=2**31 - 1), EINVAL),
                     (dict(e_local=513), EINVAL), (dict(e_local=-1), EINVAL), (dict(H=65536, F=16384), EINVAL), (dict(H=65600), EINVAL), (dict(F=65600), EINVAL),
                     (dict(logits=None), EINVAL), (dict(x=None), EINVAL), (dict(wd=None), EINVAL), (dict(out=None), EINVAL),
                     (dict(gates=None), EINVAL), (dict(x=MIS), EALIGN), (dict(res=MIS), EALIGN), (dict(ws=MIS), EALIGN),
                     (dict(ws=None), EWORKSPACE), (dict(ws_bytes=need - 1), EWORKSPACE)):
        assert call(**kw) == want, kw
    assert call(T=0, logits=None, x=None, idx=None, gates=None, out=None, ws=None, ws_bytes=0) == 0
    assert size(0, 2, 8, 128, 64) == size(65, 2, 8, 128, 64) == size(16, 2, 8, 96, 64) == size(16, 0, 8, 128, 64) == 0
    # the experts' rows in bf16 [F] and fp32 [H], of the pairs that can be local
    assert size(64, 8, 32, 7168, 2048) >= 64 * 8 * (2 * 2048 + 4 * 7168)
    assert size(64, 8, 2, 7168, 2048) >= 64 * 2 * (2 * 2048 + 4 * 7168)


def test_norm_rejects():
    call = caller("moe_layer_norm", x=FAKE, f32=0, add=None, T=4, H=128, w=None, b=None, eps=1e-5, rms=0, sum=None,
                  y=FAKE, mean=None, rstd=None)
    for kw, want in ((dict(T=-1), EINVAL), (dict(H=0), EINVAL), (dict(H=16448), EINVAL), (dict(H=96), ESHAPE),
                     (dict(f32=2), EINVAL), (dict(rms=-1), EINVAL), (dict(eps=-1e-5), EINVAL), (dict(eps=float("nan")), EINVAL),
                     (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(x=MIS), EALIGN), (dict(add=MIS), EALIGN),
                     (dict(w=MIS), EALIGN), (dict(b=MIS), EALIGN), (dict(sum=MIS), EALIGN), (dict(rstd=MIS), EALIGN)):
        assert call(**kw) == want, kw
    assert call(T=0, x=None, y=None) == 0
    size = _lib.load().moe_layer_norm_backward_workspace_size
    need = size(300, 128)
    assert need > 0 and size(0, 128) == size(4, 96) == size(-1, 128) == 0
    call = caller("moe_layer_norm_backward", dy=FAKE, s=FAKE, f32=0, T=300, H=128, w=None, mean=FAKE, rstd=FAKE, rms=0,
                  d_sum=None, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, ws_bytes=need)
    for kw, want in ((dict(T=-1), EINVAL), (dict(H=16448), EINVAL), (dict(H=96), ESHAPE), (dict(rms=1), EINVAL),
                     (dict(rms=2), EINVAL), (dict(dy=None), EINVAL), (dict(s=None), EINVAL), (dict(mean=None), EINVAL),
                     (dict(rstd=None), EINVAL), (dict(dx=None), EINVAL), (dict(d_sum=MIS), EALIGN), (dict(dw=MIS), EALIGN),
                     (dict(ws=MIS), EALIGN), (dict(ws=None), EWORKSPACE), (dict(ws_bytes=need - 1), EWORKSPACE),
                     (dict(ws=None, db=None), EWORKSPACE), (dict(ws=None, dw=None), EWORKSPACE)):
        assert call(**kw) == want, kw


def test_linear_rejects():
    lib = _lib.load()
    need = lib.moe_linear_workspace_size(1, 7168, 64)
    assert need > 0
    call = caller("moe_linear", x=FAKE, T=1, Kd=7168, w=FAKE, N=64, b=None, act=0, res=None, z=None, y=FAKE, ws=FAKE,
                  ws_bytes=need)
    for kw, want in ((dict(T=-1), EINVAL), (dict(T=2**30 + 1), EINVAL), (dict(Kd=96), ESHAPE), (dict(N=32), ESHAPE),
                     (dict(Kd=0), EINVAL), (dict(act=4), EINVAL), (dict(act=-1), EINVAL), (dict(Kd=16384, N=65536), EINVAL),
                     (dict(Kd=2**22, N=64), EINVAL), (dict(T=2**28, Kd=4096), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL),
                     (dict(b=MIS), EALIGN), (dict(res=MIS), EALIGN), (dict(z=MIS), EALIGN), (dict(y=MIS), EALIGN),
                     (dict(ws=None), EWORKSPACE), (dict(ws_bytes=need - 1), EWORKSPACE)):
        assert call(**kw) == want, kw
    assert call(T=0, x=None, w=None, y=None, ws=None, ws_bytes=0) == 0
    need = lib.moe_linear_backward_workspace_size(512, 128, 64)
    assert need > 0
    call = caller("moe_linear_backward", dy=FAKE, x=FAKE, T=512, Kd=128, w=FAKE, N=64, act=2, z=FAKE, dz=FAKE, dx=FAKE,
                  dw=FAKE, db=FAKE, ws=FAKE, ws_bytes=need)
    for kw, want in ((dict(T=-1), EINVAL), (dict(N=96), ESHAPE), (dict(act=9), EINVAL), (dict(dy=None), EINVAL),
                     (dict(z=None), EINVAL), (dict(dz=None), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL),
                     (dict(dw=MIS), EALIGN), (dict(dz=MIS), EALIGN), (dict(ws=None), EWORKSPACE),
                     (dict(ws_bytes=need - 1), EWORKSPACE), (dict(ws=None, dw=None), EWORKSPACE)):
        assert call(**kw) == want, kw
    assert lib.moe_linear_workspace_size(0, 128, 64) == lib.moe_linear_workspace_size(4, 96, 64) == 0


def test_workspaces_stay_within_what_their_operands_take():
    """Chunks of a contraction only where they leave the partial sums small beside the operands or the rows few."""
    for T in (1, 7, 64, 65, 200, 256, 257, 1000, 4001, 16384, 131072):
        for Kd, N in ((64, 64), (2048, 768), (768, 2048), (7168, 2048), (2048, 7168), (7168, 256)):
            operands = 2 * (T * Kd + Kd * N + T * N)
            assert _lib.moe_linear_workspace_size(T, Kd, N) <= max(32 * operands, 1 << 20), (T, Kd, N)
            assert _lib.moe_linear_backward_workspace_size(T, Kd, N) <= max(256 * operands, 1 << 20), (T, Kd, N)


CALLS = {
    "few": lambda s: _lib.moe_layer_few(z(4, 8, dtype=F32), z(4, 64), 2, 0, z(8, 64, 64), z(8, 64, 64), z(8, 64, 64),
                                        stream=s),
    "norm": lambda s: _lib.moe_layer_norm(z(4, 64), z(64, dtype=F32), z(64, dtype=F32), add=z(4, 64), stream=s),
    "norm_backward": lambda s: _lib.moe_layer_norm_backward(z(4, 64), z(4, 64), None, z(4, dtype=F32), z(4, dtype=F32),
                                                            stream=s),
    "linear": lambda s: _lib.moe_linear(z(4, 64), z(64, 64), act="gelu", want_z=True, stream=s),
    "linear_backward": lambda s: _lib.moe_linear_backward(z(4, 64), z(4, 64), z(64, 64), act="gelu", z=z(4, 64), stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_buffers_of_calls_with_a_stream(name, monkeypatch):
    check(Traced(monkeypatch), CALLS[name])


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 64, dtype=BF), torch.zeros(8, 64, 64, dtype=BF)
    for call in (lambda: _lib.moe_layer_norm(x), lambda: _lib.moe_linear(x, w[0]),
                 lambda: _lib.moe_layer_few(x.float()[:, :8].contiguous(), x, 2, 0, w, w, w),
                 lambda: _lib.moe_linear_backward(x, x, w[0]), lambda: _lib.moe_layer_norm_backward(x, x, None, None, None)):
        with pytest.raises(_lib.MoeError):
            call()


def test_few_buffers():
    shape = synth.WORKLOADS["tiny"].scaled(T=64)
    buf = pipeline.FewBuffers.allocate(shape, device="cpu")
    assert buf.out.shape == (64, shape.H) and buf.topk_idx.shape == buf.gates.shape == (64, shape.K)
    assert buf.ws.numel() >= _lib.moe_layer_few_workspace_size(64, shape.K, shape.EL, shape.H, shape.F)
    with pytest.raises(_lib.MoeError):
        pipeline.FewBuffers.allocate(shape.scaled(T=65), device="cpu")
