"""The calls around the experts (moe_layer_few, moe_layer_norm, moe_linear, block.py) at the edges of their arguments, on
the host."""
import pytest

from routing_permute_groupgemm_amd import _lib, block, synth
from test_block_calls_cpu import EALIGN, EINVAL, ESHAPE, EWORKSPACE, FAKE, MIS, caller
from test_stream_argument_cpu import F32, Traced, check, z


@pytest.mark.parametrize("Kd,N", [(64, 64), (2048, 64), (2112, 64), (7168, 2048), (2048, 7168), (1 << 21, 64)])
def test_plans_of_the_dense_product_without_rows(Kd, N):
    """moe_linear_backward of no rows still writes dw and db, so its size function is asked."""
    assert _lib.moe_linear_workspace_size(0, Kd, N) == 0
    assert _lib.moe_linear_backward_workspace_size(0, Kd, N) == 0


def test_block_of_no_tokens_is_allocated():
    shape = synth.WORKLOADS["tiny"].scaled(T=0, H=192, F=128, E=64, K=3, backward=True)
    b = block.BlockBuffers.allocate(shape, shared=2112, device="cpu")
    assert b.out.shape == (0, 192) and b.grads["shared_down"].shape == (1, 2112, 192)


def test_router_bias_backward_rejects():
    size = _lib.load().moe_router_bias_backward_workspace_size
    need = size(300, 128)
    assert need > 0 and size(0, 128) == size(32, 128) == size(-1, 128) == size(300, 96) == size(300, 4160) == 0
    call = caller("moe_router_bias_backward", dlogits=FAKE, T=300, E=128, dbias=FAKE, ws=FAKE, ws_bytes=need)
    for kw, want in ((dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(E=4160), EINVAL), (dict(E=96), ESHAPE),
                     (dict(dlogits=None), EINVAL), (dict(dbias=None), EINVAL), (dict(dlogits=MIS), EALIGN),
                     (dict(dbias=MIS), EALIGN), (dict(ws=MIS), EALIGN), (dict(ws=None), EWORKSPACE),
                     (dict(ws_bytes=need - 1), EWORKSPACE)):
        assert call(**kw) == want, kw


def test_buffers_of_the_router_bias_gradient_with_a_stream(monkeypatch):
    check(Traced(monkeypatch), lambda s: _lib.moe_router_bias_backward(z(4, 64, dtype=F32), stream=s))


@pytest.mark.parametrize("T,K,EL,H,F", [(1, 1, 1, 64, 64), (64, 8, 32, 7168, 2048), (64, 8, 2, 7168, 2048),
                                        (64, 16, 512, 64, 65536), (23, 8, 128, 2048, 768)])
def test_few_workspace_holds_both_values_of_h(T, K, EL, H, F):
    """Of every pair that can be local: h in two bf16 values, and the expert's row in fp32."""
    rows = T * min(K, EL)
    size = _lib.moe_layer_few_workspace_size(T, K, EL, H, F)
    assert rows * (4 * F + 4 * H) <= size <= rows * (4 * F + 4 * H) + (1 << 16)


def test_partial_sums_of_the_dense_product_are_a_few_times_its_operands():
    """A chunk of a contraction is at least 256 values deep and there are about as many workgroups as CUs, which leaves the
    partial sums at up to 2.8 times the operands (1000 x 1024 x 1024 backward); none for no rows."""
    widths = (64, 192, 768, 1024, 2048, 4096, 7168)
    for Kd in widths:
        for N in widths:
            assert _lib.moe_linear_backward_workspace_size(0, Kd, N) == 0
            for T in (1, 2, 17, 33, 64, 65, 200, 256, 257, 700, 1000, 2000, 4001, 16384, 131072):
                most = max(4 * 2 * (T * Kd + Kd * N + T * N), 1 << 20)
                assert _lib.moe_linear_workspace_size(T, Kd, N) <= most, (T, Kd, N)
                assert _lib.moe_linear_backward_workspace_size(T, Kd, N) <= most, (T, Kd, N)
