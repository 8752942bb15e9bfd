"""Cases of the experts' block-scaled operators: saved activations in 8 bits (pack8, up8, bwd8) and expert
weights in 4 bits (pack4, serve4), in plain torch and through this repository's calls.

Block formats (32 values share one scale byte s; s = 255 marks a block with a NaN or an infinity):

* 8 bits, rows [rows, cols], blocks along a row: value = q * 2^(s-133), q in -127..127, s the biased exponent of
  the block's largest magnitude, at least 7.
* 4 bits, weights [E, Kd, N], blocks along the contraction Kd: value = c * 2^(s-127), c one of 0, 0.5, 1, 1.5, 2,
  3, 4, 6 with a sign bit (code 0..7 + 8 for negative), s the largest magnitude's biased exponent - 2, at least 2.
  Codes are stored as q4 [E, N/16, KT, 64, 16] with KT = ceil(Kd/128): entry [e, n/16, k/128, 16*g + n%16, 4*t + i]
  holds k = 128*kt + 32*g + 8*t + 2*i in its low four bits and the next k in its high ones; the scales as
  s4 [E, N/16, KT, 64] with the same [.., 16*g + n%16].
"""
import math

import numpy as np
import torch

own = False

# E2M1 magnitudes by code
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the smallest layer of the tests (256 tokens, top 2): one layer's saved rows, bound by latency
        {"name": "pack8_512x512", "op": "pack8", "rows": 512, "cols": 512},
        # the saved [a | b] rows of one layer of 131072 tokens, 32 of 256 experts local, F = 2048
        {"name": "pack8_126k", "op": "pack8", "rows": 125808, "cols": 4096},
        # gate/up of the smallest layer
        {"name": "up8_tiny", "op": "up8", "T": 256, "H": 128, "F": 256, "E": 8, "EL": 8, "K": 2, "zipf": 0.0},
        # gate/up of one training step of 131072 tokens, 32 of 256 experts local, mildly skewed
        {"name": "up8_128k", "op": "up8", "T": 131072, "H": 7168, "F": 2048, "E": 256, "EL": 32, "K": 8, "zipf": 0.8},
        # the backward of the smallest layer
        {"name": "bwd8_tiny", "op": "bwd8", "T": 256, "H": 128, "F": 256, "E": 8, "EL": 8, "K": 2, "zipf": 0.0},
        # the backward of one training step of 16384 tokens, all 128 experts local
        {"name": "bwd8_16k", "op": "bwd8", "T": 16384, "H": 2048, "F": 768, "E": 128, "EL": 128, "K": 8, "zipf": 0.0},
        # one small expert matrix set, and an odd number of 64-blocks along the contraction
        {"name": "pack4_8x192x256", "op": "pack4", "E": 8, "Kd": 192, "N": 256},
        # a GPU's share of a layer's gate weights, packed when a model is loaded
        {"name": "pack4_32x7168x2048", "op": "pack4", "E": 32, "Kd": 7168, "N": 2048},
        # one token of one user: eight experts with a row each
        {"name": "serve4_1", "op": "serve4", "T": 1, "H": 4096, "F": 1536, "E": 128, "EL": 128, "K": 8, "zipf": 0.0},
        # a small batch of users on a skewed router, experts with none to a dozen rows
        {"name": "serve4_23", "op": "serve4", "T": 23, "H": 2048, "F": 768, "E": 128, "EL": 128, "K": 8, "zipf": 1.2},
        # a decode batch gathered from the GPUs of an expert-parallel group: 32 of 256 experts local
        {"name": "serve4_256", "op": "serve4", "T": 256, "H": 7168, "F": 2048, "E": 256, "EL": 32, "K": 8, "zipf": 0.8},
        # the largest decode batch: experts with about 32 rows, the busiest with over 100
        {"name": "serve4_512", "op": "serve4", "T": 512, "H": 4096, "F": 1536, "E": 128, "EL": 128, "K": 8,
         "zipf": 1.2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("pack8", "up8", "bwd8", "pack4", "serve4", "serve4"))
    if op == "pack8":
        return {"op": op, "rows": _log(rng, 1, 125808), "cols": 64 * _log(rng, 1, 64)}
    if op == "pack4":
        return {"op": op, "E": _log(rng, 1, 32), "Kd": 64 * _log(rng, 1, 112), "N": 64 * _log(rng, 1, 32)}
    H, F = 64 * _log(rng, 2, 112), 64 * _log(rng, 1, 32)
    share, zipf = rng.choice((1, 2, 8)), rng.choice((0.0, 0.8, 1.2))
    most = (128 * 4096 * 1536 if op == "serve4" else 32 * 7168 * 2048) // (H * F)
    EL = max(1, min(_log(rng, 4, 256) // share, most))
    K = min(EL * share, rng.randint(1, 8))
    T = max(_log(rng, 1, 512 if op == "serve4" else 16384), -(-8 * share // K))  # a few local rows at least
    return {"op": op, "T": T, "H": H, "F": F, "E": EL * share, "EL": EL, "K": K, "zipf": zipf}


# ---- inputs ---------------------------------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _scale8(x):
    """x float32 [rows, cols] -> (x in blocks of 32, scale exponent bytes as int32)."""
    blocks = x.view(x.shape[0], -1, 32)
    return blocks, (blocks.abs().amax(-1).view(torch.int32) >> 23).clamp(min=7)


def _pow2(e):
    """2^e for whole e of -126..127, as float32."""
    return ((e + 127) << 23).view(torch.float32)


def _pack8(x):
    blocks, s = _scale8(x)
    q = (blocks * _pow2((133 - s).clamp(min=-126)).unsqueeze(-1)).round().clamp(-127, 127)
    q = torch.where((s == 255).unsqueeze(-1), torch.zeros_like(q), q)
    return q.view(x.shape).to(torch.int8), s.to(torch.uint8)


def _unpack8(q, s):
    s = s.to(torch.int32)
    step = torch.where(s == 255, torch.full_like(s, math.nan, dtype=torch.float32), _pow2((s - 133).clamp(-126, 121)))
    return (q.to(torch.float32).view(q.shape[0], -1, 32) * step.unsqueeze(-1)).view(q.shape)


def _codes4(w):
    """w float32 [E, Kd, N] -> (codes uint8 [E, Kd, N], scale bytes int32 [E, Kd/32, N])."""
    E, Kd, N = w.shape
    u = w.abs().view(E, Kd // 32, 32, N)
    m = u.amax(2).view(torch.int32) >> 23
    s = torch.where(m == 255, m, (m - 2).clamp(min=2))
    u = (u * _pow2((127 - s).clamp(min=-126)).unsqueeze(2)).view(E, Kd, N)
    c = torch.zeros_like(w, dtype=torch.uint8)
    for at, odd in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        c += (u >= at) if odd else (u > at)  # a tie goes to the even code
    return c + 8 * torch.signbit(w).to(torch.uint8), s


def _layout4(codes, s):
    E, Kd, N = codes.shape
    KT = (Kd + 127) // 128
    c = torch.zeros((E, KT * 128, N), dtype=torch.uint8, device=codes.device)
    c[:, :Kd] = codes
    c = c.view(E, KT, 4, 4, 4, 2, N // 16, 16).permute(0, 6, 1, 2, 7, 3, 4, 5)
    q4 = (c[..., 0] | (c[..., 1] << 4)).reshape(E, N // 16, KT, 64, 16)
    b = torch.full((E, KT * 4, N), 2, dtype=torch.uint8, device=codes.device)
    b[:, :Kd // 32] = s.to(torch.uint8)
    return q4, b.view(E, KT, 4, N // 16, 16).permute(0, 3, 1, 2, 4).reshape(E, N // 16, KT, 64)


def _weights4(gen, E, Kd, N):
    """Packed N(0, 0.02) weights, a few experts at a time."""
    KT = (Kd + 127) // 128
    q4 = torch.empty((E, N // 16, KT, 64, 16), dtype=torch.uint8, device="cuda")
    s4 = torch.empty((E, N // 16, KT, 64), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (Kd * N))
    for lo in range(0, E, step):
        n = min(step, E - lo)
        w = (_randn(gen, n, Kd, N) * 0.02).to(torch.bfloat16).to(torch.float32)
        q4[lo:lo + n], s4[lo:lo + n] = _layout4(*_codes4(w))
    return q4, s4


def _plan(gen, case):
    """Routing of T tokens to K of E experts and the expert-grouped order of the pairs of the first EL experts."""
    T, E, EL, K = case["T"], case["E"], case["EL"], case["K"]
    logits = _randn(gen, T, E)
    if case["zipf"]:
        rank = torch.randperm(E, generator=gen, device="cuda").to(torch.float32)
        logits -= 0.13 * case["zipf"] * torch.log(rank + 1)
    top, idx = torch.topk(logits, K, dim=1)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)[:EL]
    # the framework's row capacity: every pair, or twice the local share that is expected (and some for small T)
    cap = T * K if EL == E else min(T * K, 2 * -(-T * K * EL // E) + 64)
    R = min(int(counts.sum()), cap)
    src = order[:R]
    pos = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    pos[src] = torch.arange(R, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(EL + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    active = torch.nonzero(counts).reshape(-1)
    slot_of = torch.zeros(EL, dtype=torch.int64, device="cuda")
    slot_of[active] = torch.arange(active.numel(), device="cuda")
    expert = flat[src]
    return {"R": R, "cap": cap, "src": torch.nn.functional.pad(src.to(torch.int32), (0, cap - R)),
            "pos": pos.view(T, K), "gates": torch.softmax(top, dim=1), "offsets": offsets, "counts": counts.tolist(),
            # experts that have rows; each row's place among them and among its expert's rows
            "active": active, "slot": slot_of[expert],
            "inner": torch.arange(R, device="cuda") - offsets.to(torch.int64)[expert],
            "most": int(counts.max())}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": dict(case)}
    if op == "pack8":
        # a layer's [a | b]: each about normal with the spread that the projection of N(0,1) tokens has
        st["x"] = (_randn(gen, case["rows"], case["cols"]) * 1.5).to(torch.bfloat16)
        return st
    if op == "pack4":
        st["w"] = torch.empty((case["E"], case["Kd"], case["N"]), dtype=torch.bfloat16, device="cuda")
        for e in range(case["E"]):
            st["w"][e] = (_randn(gen, case["Kd"], case["N"]) * 0.02).to(torch.bfloat16)
        return st
    p = st["plan"] = _plan(gen, case)
    H, F, EL, cap = case["H"], case["F"], case["EL"], p["cap"]

    def rows(cols, dtype=torch.bfloat16):
        return torch.zeros((cap, cols), dtype=dtype, device="cuda")

    def weight(kd, n):
        w = torch.empty((EL, kd, n), dtype=torch.bfloat16, device="cuda")
        for e in range(EL):
            w[e] = (_randn(gen, kd, n) * 0.02).to(torch.bfloat16)
        return w

    if op == "serve4":
        st["x"] = _randn(gen, case["T"], H).to(torch.bfloat16)
        st["gate"], st["up"] = _weights4(gen, EL, H, F), _weights4(gen, EL, H, F)
        st["down"] = _weights4(gen, EL, F, H)
        st["h"], st["y"] = rows(F), rows(H)
        st["out"] = torch.empty((case["T"], H), dtype=torch.bfloat16, device="cuda")
    elif op == "up8":
        x = _randn(gen, case["T"], H).to(torch.bfloat16)
        st["x_perm"] = x[(p["src"] // case["K"]).to(torch.int64)]
        st["w_gate"], st["w_up"] = weight(H, F), weight(H, F)
        st["h"], st["ab"] = rows(F), rows(2 * F)
        st["q"], st["s"] = rows(2 * F, torch.int8), rows(2 * F // 32, torch.uint8)
    else:
        st["dy"] = _randn(gen, cap, H).mul_(0.125).to(torch.bfloat16)
        st["w_down"] = weight(F, H)
        st["q"], st["s"] = rows(2 * F, torch.int8), rows(2 * F // 32, torch.uint8)
        spread = 0.02 * math.sqrt(H)
        for lo in range(0, cap, 16384):
            n = min(16384, cap - lo)
            ab = (_randn(gen, n, 2 * F) * spread).to(torch.bfloat16)
            st["q"][lo:lo + n], st["s"][lo:lo + n] = _pack8(ab.to(torch.float32))
        st["dab"], st["h"] = rows(2 * F), rows(F)
    return st


# ---- plain forms ----------------------------------------------------------------------------------------------


def _weights32(w4, active, Kd):
    """float32 [n, Kd, N] of the chosen experts from the packed layout."""
    q4, s4 = w4[0][active], w4[1][active]
    n, NT, KT = q4.shape[:3]
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=q4.device)
    c = torch.stack((q4 & 15, q4 >> 4), dim=-1).to(torch.int64)  # [n, NT, KT, 64, 16, 2]
    s = s4.to(torch.int32)
    step = torch.where(s == 255, torch.full_like(s, math.nan, dtype=torch.float32), _pow2((s - 127).clamp(-125, 126)))
    v = table[c].view(n, NT, KT, 64, 32) * step.unsqueeze(-1)
    v = v.view(n, NT, KT, 4, 16, 32).permute(0, 2, 3, 5, 1, 4)  # [n, KT, g, k, NT, 16]
    return v.reshape(n, KT * 128, NT * 16)[:, :Kd].contiguous()


def _padded(p, rows32):
    """Rows in expert order -> float32 [experts with rows, most rows, cols], zeros behind an expert's rows."""
    x = torch.zeros((p["active"].numel(), p["most"], rows32.shape[1]), dtype=torch.float32, device=rows32.device)
    x[p["slot"], p["inner"]] = rows32
    return x


def _whole(p, rows32):
    """bf16 of the plan's capacity: the rows behind the last routed one are as they were made, 0."""
    out = torch.zeros((p["cap"], rows32.shape[1]), dtype=torch.bfloat16, device=rows32.device)
    out[:p["R"]] = rows32.to(torch.bfloat16)
    return out


def _silu(a):
    return a / (1 + torch.exp(-a))


def _plain(st):
    op, case = st["op"], st["case"]
    bf = torch.bfloat16
    if op == "pack8":
        return {"values": _unpack8(*_pack8(st["x"].to(torch.float32))).to(bf)}
    if op == "pack4":
        w = st["w"].to(torch.float32)
        every = torch.arange(case["E"], device=w.device)
        return {"values": _weights32(_layout4(*_codes4(w)), every, case["Kd"]).to(bf)}
    p = st["plan"]
    R, F, at = p["R"], case["F"], (p["slot"], p["inner"])
    if op == "up8":
        x = _padded(p, st["x_perm"][:R].to(torch.float32))
        a = torch.bmm(x, st["w_gate"][p["active"]].to(torch.float32))[at]
        b = torch.bmm(x, st["w_up"][p["active"]].to(torch.float32))[at]
        ab = torch.cat((a, b), dim=1).to(bf).to(torch.float32)  # the checkpoint is one of the bf16 values
        return {"h": _whole(p, _silu(a) * b), "ab": _whole(p, _unpack8(*_pack8(ab)))}
    if op == "bwd8":
        w = st["w_down"][p["active"]].to(torch.float32).transpose(1, 2).contiguous()
        dh = torch.bmm(_padded(p, st["dy"][:R].to(torch.float32)), w)[at]
        ab = _unpack8(st["q"][:R], st["s"][:R])
        a, b = ab[:, :F], ab[:, F:]
        sg = 1 / (1 + torch.exp(-a))
        da, db = dh * b * sg * (1 + a * (1 - sg)), dh * a * sg
        return {"dab": _whole(p, torch.cat((da, db), dim=1)), "h": _whole(p, a * sg * b)}
    x = _padded(p, st["x"].to(torch.float32)[(p["src"][:R] // case["K"]).to(torch.int64)])
    a = torch.bmm(x, _weights32(st["gate"], p["active"], case["H"]))[at]
    b = torch.bmm(x, _weights32(st["up"], p["active"], case["H"]))[at]
    h = _silu(a) * b
    y = torch.bmm(_padded(p, h), _weights32(st["down"], p["active"], F))[at]
    y = torch.cat((y, torch.zeros_like(y[:1]) if R else torch.zeros((1, case["H"]), device=h.device)))
    pos = p["pos"].to(torch.int64)
    out = (y[torch.where(pos < 0, torch.full_like(pos, R), pos)] * p["gates"].unsqueeze(-1)).sum(1)
    return {"h": _whole(p, h), "y": _whole(p, y[:R]), "out": out.to(bf)}


# ---- this repository's calls ----------------------------------------------------------------------------------


def _own(st):
    from routing_permute_groupgemm_amd import _lib
    op, case = st["op"], st["case"]
    if op == "pack8":
        return {"values": _lib.moe_unpack8(*_lib.moe_pack8(st["x"]))}
    if op == "pack4":
        return {"values": _lib.moe_unpack4(*_lib.moe_pack4(st["w"]), case["Kd"])}
    p = st["plan"]
    cap = p["cap"]
    if op == "up8":
        _lib.moe_grouped_gemm_swiglu_save8(st["x_perm"], st["w_gate"], st["w_up"], p["offsets"], cap, h=st["h"],
                                           ab8=st["q"], ab8_scale=st["s"])
        _lib.moe_unpack8(st["q"], st["s"], x=st["ab"], offsets=p["offsets"])
        return {"h": st["h"], "ab": st["ab"]}
    if op == "bwd8":
        _lib.moe_grouped_gemm_swiglu_bwd8(st["dy"], st["w_down"], p["offsets"], cap, st["q"], st["s"],
                                          dab=st["dab"], h=st["h"])
        return {"dab": st["dab"], "h": st["h"]}
    _lib.moe_grouped_gemm4_swiglu(st["x"], p["src"], case["K"], st["gate"], st["up"], p["offsets"], cap, h=st["h"])
    _lib.moe_grouped_gemm4_combine(st["h"], st["down"], p["offsets"], cap, p["pos"], p["gates"], y=st["y"],
                                   out=st["out"])
    return {"h": st["h"], "y": st["y"], "out": st["out"]}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---- sizes ----------------------------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "pack8":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + 2 * (1 + 1 / 32) + 2), "flops": 4 * n}
    if op == "pack4":
        n = case["E"] * case["Kd"] * case["N"]
        return {"bytes": n * (2 + 2 * 17 / 32 + 2), "flops": 4 * n}
    T, H, F, E, EL, K = (case[k] for k in ("T", "H", "F", "E", "EL", "K"))
    R = T * K * EL / E                                # rows expected on the local experts
    experts = EL * (1 - (1 - K / E) ** T)             # experts expected to have one
    saved = 2 * F * (1 + 1 / 32)                      # bytes of a row's 8-bit [a | b]
    if op == "up8":
        return {"bytes": R * (2 * H + 2 * F + 2 * saved + 4 * F) + experts * 4 * H * F, "flops": 4 * R * H * F}
    if op == "bwd8":
        return {"bytes": R * (2 * H + saved + 4 * F + 2 * F) + experts * 2 * H * F, "flops": 2 * R * H * F}
    tokens = T * (1 - (1 - EL / E) ** K)              # tokens expected to have a local expert
    rows = tokens * 2 * H + 2 * R * (2 * F + 2 * H) + 2 * T * H
    return {"bytes": experts * 3 * H * F * 17 / 32 + rows, "flops": 6 * R * H * F}


# ---- from the definition, in 64 bits --------------------------------------------------------------------------


def _two(e):
    """2^e for whole e, in float64 (built from its bits: a power function may be off by a rounding)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round8(x):
    """The values that 8-bit blocks of float64 rows stand for."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().max(dim=2, keepdim=True).values
    e = torch.frexp(top).exponent - 1                 # floor(log2), of 0: -1
    e = torch.where(top > 0, e, torch.full_like(e, -120)).clamp(min=-120)
    step = _two(e - 6)
    v = torch.round(b / step).clamp(-127, 127) * step
    return torch.where(torch.isfinite(b).all(dim=2, keepdim=True), v, torch.full_like(v, math.nan)).reshape(x.shape)


def _round4(w):
    """The values that 4-bit blocks along the first axis of float64 [Kd, N] stand for."""
    b = w.reshape(-1, 32, w.shape[1])
    top = b.abs().max(dim=1, keepdim=True).values
    e = torch.where(top > 0, torch.frexp(top).exponent - 1, torch.full_like(top, -123, dtype=torch.int32))
    e = e.clamp(min=-123)
    u = b.abs() * _two(2 - e)                         # below 8
    gap = _two(torch.frexp(u).exponent.clamp(min=1) - 2)
    v = (torch.round(u / gap) * gap).clamp(max=6) * _two(e - 2) * torch.sign(b)
    return v.reshape(w.shape)


def _read4(w4, e, Kd):
    """float64 [Kd, N] of expert e of the packed weights."""
    q, s = w4[0][e].to(torch.int64), w4[1][e].to(torch.int64)
    NT, KT = q.shape[:2]
    out = torch.empty((KT, 4, 16, 2, NT, 16), dtype=torch.float64, device=q.device)  # k = 128 kt + 32 g + 2 j + nibble
    for half in (0, 1):
        c = (q >> (4 * half)) & 15
        e2, m = (c >> 1) & 3, (c & 1).to(torch.float64)
        mag = torch.where(e2 == 0, m * 0.5, (1 + 0.5 * m) * _two(e2 - 1))
        v = torch.where(c >= 8, -mag, mag) * _two(s - 127).unsqueeze(-1)            # [NT, KT, 64, 16]
        out[:, :, :, half] = v.view(NT, KT, 4, 16, 16).permute(1, 2, 4, 0, 3)
    return out.reshape(KT * 128, NT * 16)[:Kd]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "pack8":
        return {"values": _round8(st["x"].to(f64))}
    if op == "pack4":
        return {"values": torch.stack([_round4(w.to(f64)) for w in st["w"]])}
    p = st["plan"]
    R, F = p["R"], case["F"]
    ends = np.minimum(np.concatenate([[0], np.cumsum(p["counts"])]), R).tolist()
    spans = [(j, ends[j], ends[j + 1]) for j in range(case["EL"]) if ends[j + 1] > ends[j]]

    def new(cols):
        return torch.zeros((p["cap"], cols), dtype=f64, device="cuda")

    if op == "up8":
        h, ab = new(F), new(2 * F)
        for j, lo, hi in spans:
            x = st["x_perm"][lo:hi].to(f64)
            a, b = x @ st["w_gate"][j].to(f64), x @ st["w_up"][j].to(f64)
            h[lo:hi] = a * torch.sigmoid(a) * b
            ab[lo:hi] = _round8(torch.cat((a, b), 1).to(torch.bfloat16).to(f64))
        return {"h": h, "ab": ab}
    if op == "bwd8":
        dab, h = new(2 * F), new(F)
        for j, lo, hi in spans:
            dh = st["dy"][lo:hi].to(f64) @ st["w_down"][j].to(f64).t()
            step = _two(st["s"][lo:hi].to(torch.int64) - 133)
            a, b = (st["q"][lo:hi].to(f64) * step.repeat_interleave(32, dim=1)).split(F, dim=1)
            sg = torch.sigmoid(a)
            dab[lo:hi, :F] = dh * b * (sg + a * sg * (1 - sg))
            dab[lo:hi, F:] = dh * a * sg
            h[lo:hi] = a * sg * b
        return {"dab": dab, "h": h}
    h, y = new(F), new(case["H"])
    for j, lo, hi in spans:
        x = st["x"][(p["src"][lo:hi] // case["K"]).to(torch.int64)].to(f64)
        a, b = x @ _read4(st["gate"], j, case["H"]), x @ _read4(st["up"], j, case["H"])
        h[lo:hi] = a * torch.sigmoid(a) * b
        y[lo:hi] = h[lo:hi] @ _read4(st["down"], j, F)
    out = torch.zeros((case["T"], case["H"]), dtype=f64, device="cuda")
    pair = p["src"][:R].to(torch.int64)
    out.index_add_(0, pair // case["K"], y[:R] * p["gates"].reshape(-1)[pair].to(f64).unsqueeze(1))
    return {"h": h, "y": y, "out": out}
