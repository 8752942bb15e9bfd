"""The layer's forward and backward as a sequence of libmoe calls on one stream.

Buffers are torch device tensors allocated once per shape (`MoeBuffers`);
each step is one C-ABI call, and nothing is read back to the host.
"""
from __future__ import annotations

import dataclasses

import torch

from . import _lib
from .synth import MoeShape


@dataclasses.dataclass
class MoeBuffers:
    shape: MoeShape
    cap: int
    topk_idx: torch.Tensor
    gates: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    pos: torch.Tensor
    src: torch.Tensor
    x_perm: torch.Tensor | None  # None with zero_copy
    status: torch.Tensor
    ws: torch.Tensor
    h: torch.Tensor
    ab: torch.Tensor | None
    y: torch.Tensor | None  # None with weights4
    out: torch.Tensor
    # backward
    dy_perm: torch.Tensor | None = None
    dab: torch.Tensor | None = None
    dx_perm: torch.Tensor | None = None
    dx: torch.Tensor | None = None
    dw_gate: torch.Tensor | None = None
    dw_up: torch.Tensor | None = None
    dw_down: torch.Tensor | None = None
    dgates: torch.Tensor | None = None
    dlogits: torch.Tensor | None = None
    # zero-copy dispatch: the permutation is index-only, and the gate/up
    # GroupGEMM and the gate/up weight gradient read x[src[r] // K]
    zero_copy: bool = False
    # 8-bit checkpoint: the forward saves (a, b) in 8-bit blocks instead of ab, and the backward recomputes
    # h from them, so h is scratch that layers may share (allocate's h)
    checkpoint8: bool = False
    # 4-bit weights (forward4): the experts' rows stay in fp32 in ws4, there is no y
    weights4: bool = False
    ws4: torch.Tensor | None = None
    ab8: torch.Tensor | None = None
    ab8_scale: torch.Tensor | None = None

    @classmethod
    def allocate(cls, shape: MoeShape, cap: int | None = None, device="cuda", backward=None, zero_copy=False,
                 checkpoint8=False, weights4=False, h: torch.Tensor | None = None):
        """h: a buffer to use as buf.h, bf16 [at least cap, F], that layers run in turn on one stream may share:
        with checkpoint8 or without a backward, where nothing is kept in h between two steps."""
        if weights4 and (backward or checkpoint8):
            raise _lib.MoeError("allocate: 4-bit weights are for the forward only, without backward or checkpoint8")
        backward = shape.backward if backward is None else backward
        if weights4:  # serving: the products read the tokens through src
            backward, zero_copy = False, True
        T, H, F, K, EL = shape.T, shape.H, shape.F, shape.K, shape.EL
        if cap is None:
            # shape.cap is twice a share's expected rows, which a few tokens exceed now and then (one token on 32 of
            # 256 experts, top 8: 1 step in 15).  A decode step keeps room for every pair that can be local instead;
            # its rows are few
            cap = T * min(K, EL) if weights4 else shape.cap
        capn = max(cap, 1)
        if h is not None:
            if backward and not checkpoint8:
                raise _lib.MoeError("h: the backward reads it unless checkpoint8 is set, so layers cannot share it")
            if (h.dtype != torch.bfloat16 or not h.is_contiguous() or h.device.type != torch.device(device).type
                    or h.dim() != 2 or h.shape[0] < cap or h.shape[1] != F):
                raise _lib.MoeError(f"h: expected a contiguous bfloat16 tensor of at least {cap} rows of {F} columns on "
                                    f"{device}, got {h.dtype} {tuple(h.shape)} on {h.device}")
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
        ws_bytes = max(_lib.moe_permute_workspace_size(T, K, EL), 256)
        b = cls(shape=shape, cap=cap,
                topk_idx=e((T, K), dt=torch.int32), gates=e((T, K), dt=torch.float32),
                counts=e(max(EL, 1), dt=torch.int32), offsets=e(EL + 1, dt=torch.int32),
                pos=e((T, K), dt=torch.int32), src=e(capn, dt=torch.int32),
                x_perm=None if zero_copy else e((capn, H)),
                status=e(4, dt=torch.int32), ws=e(ws_bytes, dt=torch.uint8),
                h=e((capn, F)) if h is None else h,
                ab=e((capn, 2 * F)) if backward and not checkpoint8 else None,
                y=None if weights4 else e((capn, H)), out=e((T, H)), zero_copy=zero_copy,
                checkpoint8=checkpoint8 and backward, weights4=weights4)
        if weights4:
            b.ws4 = e(max(_lib.moe_gemm4_combine_workspace_size(cap, H), 256), dt=torch.uint8)
        if b.checkpoint8:
            b.ab8 = e((capn, 2 * F), dt=torch.int8)
            b.ab8_scale = e((capn, 2 * F // 32), dt=torch.uint8)
        if backward:
            b.dy_perm = e((capn, H))
            b.dab = e((capn, 2 * F))
            b.dx_perm = e((capn, H))
            b.dx = e((T, H))
            b.dw_gate = e((EL, H, F), dt=torch.float32)
            b.dw_up = e((EL, H, F), dt=torch.float32)
            b.dw_down = e((EL, F, H), dt=torch.float32)
            b.dgates = e((T, K), dt=torch.float32)
            b.dlogits = e((T, shape.E), dt=torch.float32)
        return b


def route(buf: MoeBuffers, logits):
    _lib.moe_route(logits, buf.shape.K, buf.topk_idx, buf.gates)


def permute(buf: MoeBuffers, x):
    s = buf.shape
    _lib.moe_permute(buf.topk_idx, s.e_begin, s.EL, x, buf.cap,
                     out=dict(counts=buf.counts, offsets=buf.offsets, pos=buf.pos, src=buf.src,
                              x_perm=buf.x_perm, status=buf.status), ws=buf.ws, copy_rows=not buf.zero_copy)


def expert_up(buf: MoeBuffers, w_gate, w_up, x=None):
    """x (the token rows) is needed with zero_copy only."""
    if buf.checkpoint8:
        if buf.zero_copy:
            _lib.moe_grouped_gemm_swiglu_gather_save8(x, buf.src, buf.shape.K, w_gate, w_up, buf.offsets, buf.cap,
                                                      h=buf.h, ab8=buf.ab8, ab8_scale=buf.ab8_scale)
        else:
            _lib.moe_grouped_gemm_swiglu_save8(buf.x_perm, w_gate, w_up, buf.offsets, buf.cap, h=buf.h,
                                               ab8=buf.ab8, ab8_scale=buf.ab8_scale)
    elif buf.zero_copy:
        _lib.moe_grouped_gemm_swiglu_gather(x, buf.src, buf.shape.K, w_gate, w_up, buf.offsets, buf.cap,
                                            h=buf.h, ab_save=buf.ab)
    else:
        _lib.moe_grouped_gemm_swiglu(buf.x_perm, w_gate, w_up, buf.offsets, buf.cap, h=buf.h, ab_save=buf.ab)


def _no_weights4(buf, call):
    if buf.weights4:
        raise _lib.MoeError(f"{call}: these buffers are for 4-bit weights (forward4)")


def expert_down(buf: MoeBuffers, w_down):
    _no_weights4(buf, "expert_down")
    s = buf.shape
    _lib.moe_grouped_gemm(buf.h, w_down, None, 0, buf.offsets, s.F, s.H, buf.cap, buf.y)


def combine(buf: MoeBuffers):
    _no_weights4(buf, "combine")
    _lib.moe_combine(buf.y, buf.pos, buf.gates, out=buf.out)


def forward(buf: MoeBuffers, inp: dict):
    """inp: device tensors logits, x, w_gate, w_up, w_down."""
    _no_weights4(buf, "forward")
    route(buf, inp["logits"])
    permute(buf, inp["x"])
    expert_up(buf, inp["w_gate"], inp["w_up"], inp["x"])
    expert_down(buf, inp["w_down"])
    combine(buf)
    return buf.out


def pack_weights4(inp: dict) -> dict:
    """The experts' weights in 4-bit blocks, once per model: (q4, s4) pairs for forward4."""
    return {k + "4": _lib.moe_pack4(inp[k]) for k in ("w_gate", "w_up", "w_down")}


def forward4(buf: MoeBuffers, inp: dict):
    """The forward of a decode step on 4-bit weights. inp: device tensors logits and x, and pack_weights4's
    pairs; buffers allocated with weights4=True, whose own capacity holds every local pair (with a smaller one
    given, the pairs beyond it are dropped and buf.status says so, as in forward).  At most 262140 tokens."""
    s = buf.shape
    if not buf.weights4:
        raise _lib.MoeError("forward4: the buffers need weights4=True")
    route(buf, inp["logits"])
    permute(buf, inp["x"])
    _lib.moe_grouped_gemm4_swiglu(inp["x"], buf.src, s.K, inp["w_gate4"], inp["w_up4"], buf.offsets, buf.cap, h=buf.h)
    _lib.moe_grouped_gemm4_combine(buf.h, inp["w_down4"], buf.offsets, buf.cap, buf.pos, buf.gates, out=buf.out,
                                   ws=buf.ws4)
    return buf.out


@dataclasses.dataclass
class FewBuffers:
    """Buffers of forward_few: a decode step of at most _lib.MOE_FEW_TOKENS tokens."""
    shape: MoeShape
    topk_idx: torch.Tensor
    gates: torch.Tensor
    out: torch.Tensor
    ws: torch.Tensor

    @classmethod
    def allocate(cls, shape: MoeShape, device="cuda"):
        T, K = shape.T, shape.K
        if T > _lib.MOE_FEW_TOKENS:
            raise _lib.MoeError(f"FewBuffers: at most {_lib.MOE_FEW_TOKENS} tokens, got {T}")
        ws_bytes = max(_lib.moe_layer_few_workspace_size(T, K, shape.EL, shape.H, shape.F), 256)
        e = lambda *s, dt: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
        return cls(shape=shape, topk_idx=e((T, K), dt=torch.int32), gates=e((T, K), dt=torch.float32),
                   out=e((T, shape.H), dt=torch.bfloat16), ws=e(ws_bytes, dt=torch.uint8))


def forward_few(buf: FewBuffers, inp: dict, residual: torch.Tensor | None = None):
    """forward for a few tokens in two launches, from the same inputs (logits, x and the bf16 weights); residual
    (bf16 [T, H], buf.out itself too) is added before the output's one rounding."""
    s = buf.shape
    _lib.moe_layer_few(inp["logits"], inp["x"], s.K, s.e_begin, inp["w_gate"], inp["w_up"], inp["w_down"],
                       residual=residual, topk_idx=buf.topk_idx, gates=buf.gates, out=buf.out, ws=buf.ws)
    return buf.out


def backward(buf: MoeBuffers, inp: dict):
    """inp additionally holds d_out (and x, read by the zero-copy weight gradient). Needs the forward's
    ab_save, or its 8-bit (a, b), from which h is recomputed into buf.h (whatever it holds by then)."""
    if buf.dx is None:
        raise _lib.MoeError("backward: these buffers were allocated without one")
    s = buf.shape
    H, F, EL, cap = s.H, s.F, s.EL, buf.cap
    _lib.moe_gather_gate_grad(inp["d_out"], buf.pos, buf.gates, buf.y, buf.dy_perm, buf.dgates)
    _lib.moe_route_backward(buf.topk_idx, buf.gates, buf.dgates, s.E, buf.dlogits)
    if buf.checkpoint8:
        _lib.moe_grouped_gemm_swiglu_bwd8(buf.dy_perm, inp["w_down"], buf.offsets, cap, buf.ab8, buf.ab8_scale,
                                          dab=buf.dab, h=buf.h)
    else:
        _lib.moe_grouped_gemm(buf.dy_perm, inp["w_down"], None, 1, buf.offsets, H, F, cap, buf.dab,
                              epilogue=_lib.MOE_EPI_SWIGLU_BWD, ab=buf.ab)
    _lib.moe_grouped_gemm(buf.dab, inp["w_gate"], inp["w_up"], 1, buf.offsets, F, H, cap, buf.dx_perm)
    _lib.moe_combine(buf.dx_perm, buf.pos, None, out=buf.dx)
    if buf.zero_copy:
        _lib.moe_wgrad_gate_up_gather(inp["x"], buf.src, s.K, buf.dab, buf.offsets, EL, cap, dw_gate=buf.dw_gate,
                                      dw_up=buf.dw_up)
    else:
        _lib.moe_wgrad_gate_up(buf.x_perm, buf.dab, buf.offsets, EL, cap, dw_gate=buf.dw_gate, dw_up=buf.dw_up)
    _lib.moe_wgrad(buf.h, F, buf.dy_perm, H, buf.offsets, EL, F, H, cap, dw=buf.dw_down)
    return buf.dx


def to_device(inp: dict, device="cuda") -> dict:
    """numpy inputs from synth.make_inputs -> device tensors (bf16 bit patterns viewed as bf16)."""
    import numpy as np
    out = {}
    for k, v in inp.items():
        t = torch.from_numpy(np.ascontiguousarray(v))
        if v.dtype == np.uint16:
            t = t.view(torch.int16).view(torch.bfloat16)
        out[k] = t.to(device)
    return out


def to_numpy_bits(t: torch.Tensor):
    """Device bf16 tensor -> numpy uint16 bit patterns (other dtypes: plain numpy)."""
    t = t.detach().cpu()
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).numpy().view("uint16")
    return t.numpy()
