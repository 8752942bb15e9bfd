"""Calls with stream= and no buffers of the caller's, beside work of the current stream on memory of the same sizes."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib

pytestmark = pytest.mark.gpu

E, H, F, T, K = 8, 512, 1024, 512, 4
ROWS = T * K


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


@pytest.fixture(scope="module")
def data():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(60)
    d = {"h": normal(gen, ROWS, F), "w": _lib.moe_pack4(normal(gen, E, F, H, std=0.05)),
         "offsets": torch.arange(0, ROWS + 1, ROWS // E, dtype=torch.int32, device="cuda"),
         "pos": torch.randperm(ROWS, generator=gen, device="cuda").to(torch.int32).view(T, K),
         "gates": torch.rand((T, K), generator=gen, device="cuda")}
    d["want"] = combine(d).clone()
    torch.cuda.synchronize()
    return d


def combine(d, stream=None):
    return _lib.moe_grouped_gemm4_combine(d["h"], d["w"], d["offsets"], ROWS, d["pos"], d["gates"], stream=stream)


def test_results_meet_no_earlier_work_of_the_current_stream(data):
    """The current stream has still to write the memory that it has just given back."""
    s = torch.cuda.Stream()
    old = [torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    old += [torch.empty(4 * ROWS * H, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda._sleep(20_000_000)
    for t in old:
        t.fill_(7)
    del old, t
    out = combine(data, s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, data["want"])


def test_workspaces_of_calls_that_overlap(data):
    """Calls on two streams at once, and allocations of the workspace's size on the current stream meanwhile."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(8):
        for s in streams:
            outs.append(combine(data, s))
            torch.full((4 * ROWS * H,), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, data["want"])


def test_a_result_dropped_while_the_current_stream_reads_it(data):
    """Read after waiting for the other stream, dropped before the read has run, and asked for again there."""
    s = torch.cuda.Stream()
    out = combine(data, s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    copy = out.clone()
    del out
    with torch.cuda.stream(s):
        again = [torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, data["want"]) and all((t == 7.0).all() for t in again)


def test_layer_calls_with_a_workspace_of_their_own(data):
    """The split weight gradient and the router's backward on two streams at once, without buffers."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(61)
    a, b = normal(gen, ROWS, H), normal(gen, ROWS, F)
    x, w_r = normal(gen, T, H), normal(gen, H, 64, std=0.05)
    dlogits = torch.randn((T, 64), generator=gen, device="cuda")

    def calls(stream=None):
        dw = _lib.moe_wgrad_split(a, H, b, F, data["offsets"], E, H, F, ROWS, 2, stream=stream)
        return (dw, *_lib.moe_router_backward(x, w_r, dlogits, stream=stream))

    want = calls()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            got.append(calls(s))
            torch.full((E * 2 * H * F,), 7.0, device="cuda")
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))


def test_captured_on_a_stream_of_its_own(data):
    """A call that the captured stream hands to another one, with buffers of its own; replays between eager work."""
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    combine(data, s)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        outs = [combine(data, s), combine(data, s)]
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        again = combine(data, s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, data["want"]) for out in outs + [again])
