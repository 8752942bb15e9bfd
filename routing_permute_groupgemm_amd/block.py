"""A transformer block's feed-forward half on one stream: layer norm of the residual stream, router, the local experts
(pipeline.py), and optionally a shared expert whose down product is added onto theirs.

    s = x + add,  y = norm(s),  out = experts(y) + shared(y)

The next block takes s as its x and out as its add.  Weights are a dict p of device tensors: norm_weight fp32 [H],
norm_bias fp32 [H] (without it the norm is of the root mean square), w_r bf16 [H, E] and optionally router_bias fp32 [E],
the experts' w_gate, w_up [E_L, H, F] and w_down [E_L, F, H], and with a shared expert shared_gate, shared_up [1, H, Fs]
and shared_down [1, Fs, H].
"""
from __future__ import annotations

import dataclasses

import torch

from . import _lib, pipeline
from .synth import MoeShape


@dataclasses.dataclass
class BlockBuffers:
    shape: MoeShape
    shared: int  # Fs, 0 without a shared expert
    layer: pipeline.MoeBuffers | pipeline.FewBuffers
    y: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    logits: torch.Tensor
    ws: torch.Tensor  # one call's scratch after the other
    out: torch.Tensor
    sum: torch.Tensor | None = None
    s: torch.Tensor | None = None  # the last forward's residual stream: its x, or sum
    one: torch.Tensor | None = None  # the shared expert's row offsets: all tokens
    h: torch.Tensor | None = None
    ab: torch.Tensor | None = None
    # backward: the three gradients of y next to each other, and the rows that make a token's sum
    parts: torch.Tensor | None = None
    pos: torch.Tensor | None = None
    dy: torch.Tensor | None = None
    dab: torch.Tensor | None = None
    grads: dict | None = None  # buffers of every gradient; backward returns those that there are

    @classmethod
    def allocate(cls, shape: MoeShape, shared=0, device="cuda", backward=None, few=False, x_dtype=torch.bfloat16,
                 cap: int | None = None):
        """few: a decode step of at most _lib.MOE_FEW_TOKENS tokens in the few-token form; x_dtype: the residual
        stream's type, bf16 or fp32; cap: the rows that the experts' buffers hold, as MoeBuffers.allocate's: on a share of
        the experts twice the expected rows unless it is given, pairs beyond it are dropped and layer.status says so
        (T * min(K, EL) holds every pair; the few-token form always does)."""
        if few and backward:
            raise _lib.MoeError("allocate: the few-token form is for the forward only")
        if few and cap is not None:
            raise _lib.MoeError("allocate: the few-token form has no capacity")
        backward = False if few else shape.backward if backward is None else backward
        T, H, E = shape.T, shape.H, shape.E
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
        need = [256, _lib.moe_router_workspace_size(T, H, E)]
        if shared:
            need.append(_lib.moe_linear_workspace_size(T, shared, H))
        if backward:
            need.append(_lib.moe_layer_norm_backward_workspace_size(T, H))
            need.append(_lib.moe_router_bias_backward_workspace_size(T, E))
            if shared:
                need.append(_lib.moe_linear_backward_workspace_size(T, shared, H))
        layer = (pipeline.FewBuffers.allocate(shape, device) if few else
                 pipeline.MoeBuffers.allocate(shape, cap=cap, device=device, backward=backward))
        b = cls(shape=shape, shared=shared, layer=layer, y=e((T, H)), mean=e(T, dt=torch.float32),
                rstd=e(T, dt=torch.float32), logits=e((T, E), dt=torch.float32), ws=e(max(need), dt=torch.uint8),
                out=e((T, H)) if shared else layer.out, sum=e((T, H), dt=x_dtype))
        if shared:
            b.one = torch.tensor([0, T], dtype=torch.int32, device=device)
            b.h = e((T, shared))
            b.ab = e((T, 2 * shared)) if backward else None
        if backward:
            n = 3 if shared else 2
            b.parts = e((n * T, H))
            b.layer.dx = b.parts[:T]
            b.pos = torch.stack([torch.arange(T, dtype=torch.int32, device=device) + i * T for i in range(n)], 1)
            b.pos = b.pos.contiguous()
            b.dy = e((T, H))
            b.dab = e((T, 2 * shared)) if shared else None
            f32 = lambda *s: e(s, dt=torch.float32)  # noqa: E731
            b.grads = {"x": e((T, H), dt=x_dtype), "norm_weight": f32(H), "norm_bias": f32(H), "w_r": f32(H, E),
                       "router_bias": f32(E), "w_gate": layer.dw_gate, "w_up": layer.dw_up, "w_down": layer.dw_down}
            if shared:
                b.grads.update(shared_gate=f32(1, H, shared), shared_up=f32(1, H, shared), shared_down=f32(1, shared, H))
        return b


def forward(b: BlockBuffers, p: dict, x: torch.Tensor, add: torch.Tensor | None = None, eps=1e-5):
    """x: the residual stream [T, H]; add (bf16): what is added to it first -> (s, out), out the bf16 sum of the experts."""
    rms = p.get("norm_bias") is None
    b.s, _, _, _ = _lib.moe_layer_norm(x, p["norm_weight"], p.get("norm_bias"), add=add, eps=eps, rms=rms,
                                       sum=None if add is None else b.sum, y=b.y, mean=None if rms else b.mean, rstd=b.rstd)
    _lib.moe_router_logits(b.y, p["w_r"], p.get("router_bias"), logits=b.logits, ws=b.ws)
    inp = {"logits": b.logits, "x": b.y, "w_gate": p["w_gate"], "w_up": p["w_up"], "w_down": p["w_down"]}
    few = isinstance(b.layer, pipeline.FewBuffers)
    if not few:
        pipeline.forward(b.layer, inp)
    if b.shared:
        _lib.moe_grouped_gemm_swiglu(b.y, p["shared_gate"], p["shared_up"], b.one, b.shape.T, h=b.h, ab_save=b.ab)
        _lib.moe_linear(b.h, p["shared_down"][0], residual=None if few else b.layer.out, y=b.out, ws=b.ws)
    if few:
        _lib.moe_layer_few(b.logits, b.y, b.shape.K, b.shape.e_begin, p["w_gate"], p["w_up"], p["w_down"],
                           residual=b.out if b.shared else None, topk_idx=b.layer.topk_idx, gates=b.layer.gates, out=b.out,
                           ws=b.layer.ws)
    return b.s, b.out


def backward(b: BlockBuffers, p: dict, d_out: torch.Tensor, d_s: torch.Tensor | None = None):
    """From the gradients of the forward's out (bf16) and of its s past this block (x's type) -> the gradients of x (add's
    is the same) and of the weights that p has, in b.grads' buffers.  The gates' gradients reach the router."""
    if b.grads is None:
        raise _lib.MoeError("backward: these buffers were allocated without one")
    if b.s is None:
        raise _lib.MoeError("backward: no forward was run on these buffers")
    T, H, Fs, g = b.shape.T, b.shape.H, b.shared, b.grads
    rms = p.get("norm_bias") is None
    pipeline.backward(b.layer, {"d_out": d_out, "x": b.y, "w_gate": p["w_gate"], "w_up": p["w_up"], "w_down": p["w_down"]})
    _lib.moe_router_backward(b.y, p["w_r"], b.layer.dlogits, dx=b.parts[T:2 * T], dw_r=g["w_r"], ws=b.ws)
    if p.get("router_bias") is not None:
        _lib.moe_router_bias_backward(b.layer.dlogits, dbias=g["router_bias"], ws=b.ws)
    if Fs:
        _lib.moe_grouped_gemm(d_out, p["shared_down"], None, 1, b.one, H, Fs, T, b.dab,
                              epilogue=_lib.MOE_EPI_SWIGLU_BWD, ab=b.ab)
        _lib.moe_grouped_gemm(b.dab, p["shared_gate"], p["shared_up"], 1, b.one, Fs, H, T, b.parts[2 * T:])
        _lib.moe_wgrad_gate_up(b.y, b.dab, b.one, 1, T, dw_gate=g["shared_gate"], dw_up=g["shared_up"])
        _lib.moe_linear_backward(d_out, b.h, p["shared_down"][0], want_dx=False, want_db=False, dw=g["shared_down"][0],
                                 ws=b.ws)
    _lib.moe_combine(b.parts, b.pos, None, out=b.dy)
    _lib.moe_layer_norm_backward(b.dy, b.s, p["norm_weight"], None if rms else b.mean, b.rstd, d_sum=d_s, rms=rms,
                                 dx=g["x"], dw=g["norm_weight"], db=None if rms else g["norm_bias"], ws=b.ws)
    return {k: v for k, v in g.items() if k == "x" or p.get(k) is not None}
