"""Calls with stream=: every buffer that the binding makes itself comes from that stream's memory, and results are
recorded for the caller's stream.  The library and the streams are stand-ins here; nothing is launched."""
import contextlib

import pytest
import torch

from routing_permute_groupgemm_amd import _lib

BF, F32, I32, I8, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8


class Stream:
    device_index = -1
    cuda_stream = 0x51


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


class Traced:
    """What a call allocated: data pointer -> the stream whose memory it is (None: the current one), the pointers
    recorded for the caller's stream, and the arguments of the library's calls."""

    def __init__(self, monkeypatch):
        self.within, self.owner, self.recorded, self.calls, self.kept = None, {}, set(), [], []
        empty = torch.empty

        def traced_empty(shape, dtype, device):
            t = empty(shape, dtype=dtype)
            self.kept.append(t)
            self.owner[t.data_ptr()] = self.within
            return t

        @contextlib.contextmanager
        def on(stream):
            self.within = stream
            yield
            self.within = None

        class Lib:
            def __getattr__(lib, name):
                def call(*args):
                    self.calls.append((name, args))
                    return 512 if name.endswith("workspace_size") else 0
                return call

        monkeypatch.setattr(torch, "empty", traced_empty)
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device: "caller's")
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.recorded.add((t.data_ptr(), s)),
                            raising=False)
        monkeypatch.setattr(_lib, "load", Lib)
        # the tensors here are on the host, whose device index is -1
        monkeypatch.setattr(_lib, "_device", lambda stream, t: -1)
        monkeypatch.setattr(_lib, "_need", lambda t, dtype, name: None)


@pytest.fixture
def traced(monkeypatch):
    return Traced(monkeypatch)


def check(traced, call):
    s = Stream()
    result = call(s)
    result = result if isinstance(result, tuple) else (result,)
    assert traced.owner and all(owner is s for owner in traced.owner.values())
    for t in result:
        assert (t.data_ptr(), "caller's") in traced.recorded
    _, args = traced.calls[-1]
    assert args[-1] == s.cuda_stream
    # the buffers are the ones that the library was given
    assert set(traced.owner) <= set(args)


OFF = z(3, dtype=I32)
W4 = (z(2, 4, 1, 64, 16, dtype=U8), z(2, 4, 1, 64, dtype=U8))

BLOCK_SCALED = {
    "pack8": lambda s: _lib.moe_pack8(z(4, 64), stream=s),
    "unpack8": lambda s: _lib.moe_unpack8(z(4, 64, dtype=I8), z(4, 2, dtype=U8), stream=s),
    "save8": lambda s: _lib.moe_grouped_gemm_swiglu_save8(z(4, 64), z(2, 64, 64), z(2, 64, 64), OFF, 4, stream=s),
    "gather_save8": lambda s: _lib.moe_grouped_gemm_swiglu_gather_save8(
        z(4, 64), z(4, dtype=I32), 1, z(2, 64, 64), z(2, 64, 64), OFF, 4, stream=s),
    "bwd8": lambda s: _lib.moe_grouped_gemm_swiglu_bwd8(z(4, 64), z(2, 64, 64), OFF, 4, z(4, 128, dtype=I8),
                                                        z(4, 4, dtype=U8), stream=s),
    "pack4": lambda s: _lib.moe_pack4(z(2, 64, 64), stream=s),
    "unpack4": lambda s: _lib.moe_unpack4(*W4, 64, stream=s),
    "gemm4_swiglu": lambda s: _lib.moe_grouped_gemm4_swiglu(z(4, 64), z(4, dtype=I32), 1, W4, W4, OFF, 4, stream=s),
    "gemm4": lambda s: _lib.moe_grouped_gemm4(z(4, 64), W4, OFF, 4, stream=s),
    "gemm4_combine": lambda s: _lib.moe_grouped_gemm4_combine(z(4, 64), W4, OFF, 4, z(4, 1, dtype=I32),
                                                              z(4, 1, dtype=F32), stream=s),
}


@pytest.mark.parametrize("name", list(BLOCK_SCALED))
def test_buffers_of_the_block_scaled_calls(name, traced):
    check(traced, BLOCK_SCALED[name])


def test_a_workspace_too_small_is_replaced_on_the_stream(traced):
    small = z(16, dtype=U8)
    check(traced, lambda s: _lib.moe_grouped_gemm4_combine(z(4, 64), W4, OFF, 4, z(4, 1, dtype=I32),
                                                           z(4, 1, dtype=F32), ws=small, stream=s))
    assert len(traced.owner) == 2  # out and the workspace
    assert small.data_ptr() not in traced.calls[-1][1]


def test_without_a_stream_the_current_one_allocates(traced, monkeypatch):
    monkeypatch.setattr(_lib, "_handle", lambda stream, dev: 0x52)
    _lib.moe_pack8(z(4, 64))
    assert set(traced.owner.values()) == {None} and not traced.recorded


LAYER = {
    "route": lambda s: _lib.moe_route(z(4, 8, dtype=F32), 2, stream=s),
    "route_backward": lambda s: _lib.moe_route_backward(z(4, 2, dtype=I32), z(4, 2, dtype=F32), z(4, 2, dtype=F32), 8,
                                                        stream=s),
    "permute": lambda s: tuple(_lib.moe_permute(z(4, 2, dtype=I32), 0, 8, z(4, 64), 8, stream=s).values()),
    "swiglu": lambda s: _lib.moe_grouped_gemm_swiglu(z(4, 64), z(2, 64, 64), z(2, 64, 64), OFF, 4, stream=s),
    "swiglu_gather": lambda s: _lib.moe_grouped_gemm_swiglu_gather(z(4, 64), z(4, dtype=I32), 1, z(2, 64, 64),
                                                                   z(2, 64, 64), OFF, 4, stream=s),
    "combine": lambda s: _lib.moe_combine(z(4, 64), z(4, 1, dtype=I32), None, stream=s),
    "gather_gate_grad": lambda s: _lib.moe_gather_gate_grad(z(4, 64), z(4, 1, dtype=I32), z(4, 1, dtype=F32),
                                                            z(4, 64), z(4, 64), stream=s)[1],
    "wgrad": lambda s: _lib.moe_wgrad(z(4, 64), 64, z(4, 64), 64, OFF, 2, 64, 64, 4, stream=s),
    "wgrad_gate_up": lambda s: _lib.moe_wgrad_gate_up(z(4, 64), z(4, 128), OFF, 2, 4, stream=s),
    "wgrad_gate_up_gather": lambda s: _lib.moe_wgrad_gate_up_gather(z(4, 64), z(4, dtype=I32), 1, z(4, 128), OFF, 2, 4,
                                                                    stream=s),
    "wgrad_split": lambda s: _lib.moe_wgrad_split(z(4, 64), 64, z(4, 64), 64, OFF, 2, 64, 64, 4, 2, stream=s),
    "router_logits": lambda s: _lib.moe_router_logits(z(4, 64), z(64, 8), stream=s),
    "router_backward": lambda s: _lib.moe_router_backward(z(4, 64), z(64, 8), z(4, 8, dtype=F32), stream=s),
    "probe_mfma": lambda s: _lib.moe_probe_mfma(z(4, 8, 64, 8), 1, stream=s),
    "probe_mfma16": lambda s: _lib.moe_probe_mfma16(z(4, 16, 64, 8), 1, stream=s),
}


@pytest.mark.parametrize("name", list(LAYER))
def test_buffers_of_the_layer_calls(name, traced):
    check(traced, LAYER[name])
