"""Cases of the operators around the experts: a whole layer for a few tokens (few), layer norm with the residual
stream's addition, forward and backward (norm), and the dense product with bias, activation and residual in its
epilogue (linear), in plain torch and through this repository's calls.

few     softmax over the K best of E scores (ties to the lowest expert), renormalised over them; the pairs of the
        experts e_begin .. e_begin+EL-1 are computed here:
        out[t] = residual[t] + sum_k gate[t,k] * (silu(x_t Wg_j) * (x_t Wu_j)) Wd_j
norm    s = x + add, rounded to the residual stream's type; y = (s - mean) * rstd * weight + bias, or without mean
        and bias (rms); backward: dx = rstd * (g - avg(g) - xh * avg(g xh)) + d_sum with g = dy * weight and
        xh = (s - mean) * rstd (rms: no avg(g)), dw = sum dy xh, db = sum dy
linear  z = x w + bias, y = act(z) + residual; backward from dy and the saved bf16 z: dz = dy act'(z),
        dx = dz w^T, dw = x^T dz, db = sum dz
"""
import math

import torch

own = False

_EPS = 1e-5


def listed():
    return [
        # one token on the smallest layer of the tests: bound by latency
        {"name": "few_1_tiny", "op": "few", "T": 1, "H": 128, "F": 256, "E": 8, "e0": 0, "EL": 8, "K": 2, "zipf": 0.0,
         "res": False},
        # one token of one user: eight experts with a row each
        {"name": "few_1", "op": "few", "T": 1, "H": 4096, "F": 1536, "E": 128, "e0": 0, "EL": 128, "K": 8, "zipf": 0.0,
         "res": True},
        # a small batch of users on a skewed router: experts with none to a dozen rows
        {"name": "few_23", "op": "few", "T": 23, "H": 2048, "F": 768, "E": 128, "e0": 0, "EL": 128, "K": 8,
         "zipf": 1.2, "res": True},
        # the largest batch of this form on one GPU of an expert-parallel group: 32 of 256 experts here
        {"name": "few_64", "op": "few", "T": 64, "H": 7168, "F": 2048, "E": 256, "e0": 0, "EL": 32, "K": 8,
         "zipf": 0.8, "res": False},
        # the norm in front of a decode step's layer
        {"name": "norm_1", "op": "norm", "T": 1, "H": 7168, "f32": False, "rms": True, "add": True, "back": False},
        # a ragged small batch in training, an odd number of 64-column blocks
        {"name": "norm_127", "op": "norm", "T": 127, "H": 2112, "f32": False, "rms": False, "add": False, "back": True},
        # a training step whose residual stream is kept in fp32
        {"name": "norm_8k_f32", "op": "norm", "T": 8192, "H": 4096, "f32": True, "rms": False, "add": True,
         "back": True},
        # the largest training step: 131072 tokens
        {"name": "norm_128k", "op": "norm", "T": 131072, "H": 7168, "f32": False, "rms": True, "add": True,
         "back": True},
        # a shared expert's down product of one token, onto the routed experts' output
        {"name": "linear_1", "op": "linear", "T": 1, "Kd": 2048, "N": 7168, "act": "none", "bias": False, "res": True,
         "back": False},
        # a ragged decode batch through a dense layer's first product
        {"name": "linear_41", "op": "linear", "T": 41, "Kd": 4096, "N": 1536, "act": "gelu", "bias": True, "res": False,
         "back": False},
        # a dense feed-forward product in training on an odd number of tokens
        {"name": "linear_4001", "op": "linear", "T": 4001, "Kd": 2048, "N": 768, "act": "relu", "bias": True,
         "res": True, "back": True},
        # the shared expert's down product of the largest training step
        {"name": "linear_128k", "op": "linear", "T": 131072, "Kd": 2048, "N": 7168, "act": "none", "bias": True,
         "res": True, "back": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("few", "few", "norm", "norm", "linear", "linear"))
    if op == "few":
        H, F = 64 * _log(rng, 1, 112), 64 * _log(rng, 1, 32)
        share = rng.choice((1, 1, 2, 8))
        EL = max(1, min(_log(rng, 2, 256) // share, 32 * 7168 * 2048 // (H * F)))
        return {"op": op, "T": _log(rng, 1, 64), "H": H, "F": F, "E": EL * share, "e0": EL * rng.randrange(share),
                "EL": EL, "K": min(EL * share, rng.randint(1, 8)), "zipf": rng.choice((0.0, 0.8, 1.2)),
                "res": rng.random() < 0.5}
    if op == "norm":
        H, f32 = 64 * _log(rng, 1, 128), rng.random() < 0.4
        T = _log(rng, 1, min(131072, 131072 * 7168 // (H * (2 if f32 else 1))))
        return {"op": op, "T": T, "H": H, "f32": f32, "rms": rng.random() < 0.5, "add": rng.random() < 0.5,
                "back": rng.random() < 0.7}
    Kd, N = 64 * _log(rng, 1, 112), 64 * _log(rng, 1, 112)
    back = rng.random() < 0.5
    T = _log(rng, 1, min(131072, 131072 * 2048 * 7168 // (Kd * N * 4)))
    return {"op": op, "T": T, "Kd": Kd, "N": N, "act": rng.choice(("none", "relu", "silu", "gelu")),
            "bias": rng.random() < 0.6, "res": rng.random() < 0.5, "back": back}


# ---- inputs ---------------------------------------------------------------------------------------------------


def _bf16(gen, *shape, std=1.0):
    """Normal bf16 values, made in pieces of at most 2^28."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for lo in range(0, flat.numel(), 1 << 28):
        part = flat[lo:lo + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(std))
    return out


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, T = case["op"], case["T"]
    st = {"case": dict(case)}
    if op == "few":
        H, F, E, EL = (case[k] for k in ("H", "F", "E", "EL"))
        logits = _normal(gen, T, E)
        if case["zipf"]:  # a skewed router: a bias that falls with the logarithm of an expert's rank
            rank = torch.randperm(E, generator=gen, device="cuda").to(torch.float32)
            logits -= 0.13 * case["zipf"] * torch.log(rank + 1)
        st["logits"], st["x"] = logits, _bf16(gen, T, H)
        st["w_gate"], st["w_up"] = _bf16(gen, EL, H, F, std=0.02), _bf16(gen, EL, H, F, std=0.02)
        st["w_down"] = _bf16(gen, EL, F, H, std=0.02)
        st["res"] = _bf16(gen, T, H) if case["res"] else None
    elif op == "norm":
        H, dtype = case["H"], torch.float32 if case["f32"] else torch.bfloat16
        # a residual stream: every column with a spread and an offset of its own, a few of them large
        spread = torch.exp(0.5 * _normal(gen, H)) * torch.where(torch.arange(H, device="cuda") % 61 == 7, 8.0, 1.0)
        shift = 0.3 + 0.2 * _normal(gen, H)

        def stream():
            out = torch.empty((T, H), dtype=dtype, device="cuda")
            for lo in range(0, T, 32768):
                part = out[lo:lo + 32768]
                part.copy_(_normal(gen, *part.shape).mul_(spread).add_(shift))
            return out

        st["x"] = stream()
        st["add"] = _bf16(gen, T, H) if case["add"] else None
        st["weight"] = 1 + 0.1 * _normal(gen, H)
        st["bias"] = None if case["rms"] else 0.1 * _normal(gen, H)
        if case["back"]:
            st["dy"] = _bf16(gen, T, H, std=0.125)
            st["d_sum"] = _bf16(gen, T, H, std=0.125).to(dtype) if case["add"] else None
    else:
        Kd, N = case["Kd"], case["N"]
        st["x"], st["w"] = _bf16(gen, T, Kd), _bf16(gen, Kd, N, std=0.02)
        st["bias"] = 0.1 * _normal(gen, N) if case["bias"] else None
        st["res"] = _bf16(gen, T, N) if case["res"] else None
        if case["back"]:
            st["dy"] = _bf16(gen, T, N, std=0.125)
            # what a forward of these sizes saved: values of z's spread
            st["z"] = None if case["act"] == "none" else _bf16(gen, T, N, std=0.02 * math.sqrt(Kd))
    return st


# ---- plain forms ----------------------------------------------------------------------------------------------


def _plain_few(st):
    case = st["case"]
    K, e0, EL, T = case["K"], case["e0"], case["EL"], case["T"]
    score, order = torch.sort(st["logits"], dim=1, descending=True, stable=True)
    idx, top = order[:, :K], score[:, :K]
    ex = torch.exp(top - top[:, :1])
    gates = ex / ex.sum(1, keepdim=True)
    # the weight of each token on each local expert, and the experts that have any
    mine = torch.zeros((T, case["E"]), device=gates.device).scatter_(1, idx, gates)[:, e0:e0 + EL]
    used = torch.zeros((T, case["E"]), dtype=torch.bool, device=gates.device).scatter_(1, idx, True)[:, e0:e0 + EL]
    active = torch.nonzero(used.any(0)).reshape(-1)
    x = st["x"].to(torch.float32)
    a = torch.matmul(x, st["w_gate"][active].to(torch.float32))      # [active, T, F]
    b = torch.matmul(x, st["w_up"][active].to(torch.float32))
    y = torch.bmm(a / (1 + torch.exp(-a)) * b, st["w_down"][active].to(torch.float32))
    out = (y * mine[:, active].t().unsqueeze(2)).sum(0)
    if st["res"] is not None:
        out = out + st["res"].to(torch.float32)
    return {"out": out.to(torch.bfloat16), "idx": idx.to(torch.int32), "gates": gates}


def _plain_norm(st):
    case, dtype = st["case"], st["x"].dtype
    s = st["x"] if st["add"] is None else (st["x"].to(torch.float32) + st["add"].to(torch.float32)).to(dtype)
    v = s.to(torch.float32)
    got = {"sum": None if st["add"] is None else s}
    if not case["rms"]:
        mean = v.mean(1, dtype=torch.float64, keepdim=True).to(torch.float32)
        got["mean"] = mean.reshape(-1)
        v = v - mean
    rstd = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + _EPS)
    v = v * rstd
    y = v * st["weight"]
    got["rstd"], got["y"] = rstd.reshape(-1), (y if st["bias"] is None else y + st["bias"]).to(torch.bfloat16)
    if case["back"]:
        dy = st["dy"].to(torch.float32)
        got["dw"] = (dy * v).sum(0, dtype=torch.float64).to(torch.float32)
        g = dy * st["weight"]
        dx = g - v * (g * v).mean(1, keepdim=True)
        if not case["rms"]:
            got["db"] = dy.sum(0, dtype=torch.float64).to(torch.float32)
            dx = dx - g.mean(1, keepdim=True)
        dx = dx * rstd
        got["dx"] = (dx if st["d_sum"] is None else dx + st["d_sum"].to(torch.float32)).to(dtype)
    return got


def _act(act, z):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _slope(act, z):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _plain_linear(st):
    case = st["case"]
    act, bf = case["act"], torch.bfloat16
    w = st["w"].to(torch.float32)
    z = st["x"].to(torch.float32) @ w
    if st["bias"] is not None:
        z = z + st["bias"]
    got = {"z": z.to(bf) if case["back"] and act != "none" else None}
    y = _act(act, z)
    got["y"] = (y if st["res"] is None else y + st["res"].to(torch.float32)).to(bf)
    if case["back"]:
        dz = st["dy"].to(torch.float32)
        if act != "none":
            dz = dz * _slope(act, st["z"].to(torch.float32))
            got["dz"] = dz.to(bf)
        got["dx"] = (dz @ w.t()).to(bf)
        if act in ("none", "relu"):  # dz is a bf16 as it is; where it is rounded, dw is a product of the rounded values
            got["dw"] = st["x"].to(torch.float32).t() @ dz
        if st["bias"] is not None:
            got["db"] = dz.sum(0, dtype=torch.float64).to(torch.float32)
    return got


# ---- this repository's calls ----------------------------------------------------------------------------------


def _own(st):
    from routing_permute_groupgemm_amd import _lib
    case = st["case"]
    if case["op"] == "few":
        out, idx, gates = _lib.moe_layer_few(st["logits"], st["x"], case["K"], case["e0"], st["w_gate"], st["w_up"],
                                             st["w_down"], residual=st["res"])
        return {"out": out, "idx": idx, "gates": gates}
    if case["op"] == "norm":
        rms = case["rms"]
        s, y, mean, rstd = _lib.moe_layer_norm(st["x"], st["weight"], st["bias"], add=st["add"], eps=_EPS, rms=rms)
        got = {"sum": None if st["add"] is None else s, "y": y, "rstd": rstd}
        if not rms:
            got["mean"] = mean
        if case["back"]:
            dx, dw, db = _lib.moe_layer_norm_backward(st["dy"], s, st["weight"], mean, rstd, d_sum=st["d_sum"],
                                                      rms=rms, want_db=not rms)
            got.update({"dx": dx, "dw": dw} if rms else {"dx": dx, "dw": dw, "db": db})
        return got
    act = case["act"]
    saved = case["back"] and act != "none"
    y, z = _lib.moe_linear(st["x"], st["w"], bias=st["bias"], act=act, residual=st["res"], want_z=saved)
    got = {"y": y, "z": z}
    if case["back"]:
        dz, dx, dw, db = _lib.moe_linear_backward(st["dy"], st["x"], st["w"], act=act, z=st["z"],
                                                  want_dw=act in ("none", "relu"), want_db=st["bias"] is not None)
        got.update({"dz": dz if saved else None, "dx": dx, "dw": dw, "db": db})
    return got


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_few(state) if op == "few" else _plain_norm(state) if op == "norm" else _plain_linear(state)


# ---- sizes ----------------------------------------------------------------------------------------------------


def work(case):
    op, T = case["op"], case["T"]
    if op == "few":
        H, F, E, EL, K = (case[k] for k in ("H", "F", "E", "EL", "K"))
        experts = EL * (1 - (1 - K / E) ** T)         # local experts expected to have a token
        rows = 4 * T * E + 2 * T * H * (3 if case["res"] else 2) + 8 * T * K
        return {"bytes": experts * 6 * H * F + rows, "flops": 6 * T * K * EL / E * H * F}
    if op == "norm":
        n, size = T * case["H"], 4 if case["f32"] else 2
        moved = n * (size + (2 + size if case["add"] else 0) + 2)
        if case["back"]:
            moved += n * (2 + 2 * size + (size if case["add"] else 0))
        return {"bytes": moved, "flops": n * (22 if case["back"] else 8)}
    Kd, N, saved = case["Kd"], case["N"], case["act"] != "none"
    moved = 2 * (T * Kd + Kd * N + T * N * (2 if case["res"] else 1))
    flops = 2 * T * Kd * N
    if case["back"]:
        dw = case["act"] in ("none", "relu")
        moved += 2 * (T * Kd + Kd * N + T * N * (4 if saved else 1)) + (2 * T * Kd + 4 * Kd * N if dw else 0)
        flops *= 3 if dw else 2
    return {"bytes": moved, "flops": flops}


# ---- from the definition, in 64 bits --------------------------------------------------------------------------


def _exact_few(st):
    case = st["case"]
    T, K, e0, EL = (case[k] for k in ("T", "K", "e0", "EL"))
    out = torch.zeros((T, case["H"]), dtype=torch.float64, device="cuda")
    if st["res"] is not None:
        out += st["res"]
    host = st["logits"].double().cpu().tolist()
    idx = [sorted(range(case["E"]), key=lambda e: (-row[e], e))[:K] for row in host]
    gates = torch.stack([torch.softmax(torch.tensor([row[e] for e in chosen], dtype=torch.float64), 0)
                         for row, chosen in zip(host, idx)])
    for j in range(EL):
        pairs = [(t, k) for t in range(T) for k in range(K) if idx[t][k] == e0 + j]
        if not pairs:
            continue
        at = torch.tensor([t for t, _ in pairs], device="cuda")
        weight = torch.tensor([float(gates[t, k]) for t, k in pairs], dtype=torch.float64, device="cuda")
        x = st["x"][at].double()
        a = x @ st["w_gate"][j].double()
        h = a * torch.sigmoid(a) * (x @ st["w_up"][j].double())
        out[at] += weight[:, None] * (h @ st["w_down"][j].double())
    return {"out": out, "idx": None, "gates": gates}


def _exact_norm(st):
    case, H = st["case"], st["case"]["H"]
    names = ["y"] + (["dx"] if case["back"] else [])
    got = {k: torch.empty((case["T"], H), dtype=torch.float64, device="cuda") for k in names}
    got["rstd"] = torch.empty(case["T"], dtype=torch.float64, device="cuda")
    got["sum"] = None
    if not case["rms"]:
        got["mean"] = torch.empty_like(got["rstd"])
    sums = {k: torch.zeros(H, dtype=torch.float64, device="cuda") for k in ("dw", "db")}
    w = st["weight"].double()
    for lo in range(0, case["T"], 16384):
        at = slice(lo, lo + 16384)
        s = st["x"][at]
        if st["add"] is not None:
            s = (s.double() + st["add"][at].double()).to(s.dtype)
        s = s.double()
        mean = torch.zeros_like(s[:, :1]) if case["rms"] else s.sum(1, keepdim=True) / H
        var = (s - mean).square().sum(1, keepdim=True) / H
        rstd = (var + _EPS).rsqrt()
        xh = (s - mean) * rstd
        got["y"][at] = xh * w if st["bias"] is None else xh * w + st["bias"].double()
        got["rstd"][at] = rstd[:, 0]
        if not case["rms"]:
            got["mean"][at] = mean[:, 0]
        if case["back"]:
            dy = st["dy"][at].double()
            sums["dw"] += (dy * xh).sum(0)
            sums["db"] += dy.sum(0)
            # the derivative of sum(dy y): through xh directly, through the mean, and through the spread
            g = dy * w
            dx = rstd * g - rstd * xh * ((g * xh).sum(1, keepdim=True) / H)
            if not case["rms"]:
                dx -= rstd * (g.sum(1, keepdim=True) / H)
            got["dx"][at] = dx if st["d_sum"] is None else dx + st["d_sum"][at].double()
    if case["back"]:
        got.update({"dw": sums["dw"]} if case["rms"] else sums)
    return got


def _exact_linear(st):
    case = st["case"]
    act, T, N = case["act"], case["T"], case["N"]
    saved = case["back"] and act != "none"
    new = lambda cols: torch.empty((T, cols), dtype=torch.float64, device="cuda")  # noqa: E731
    got = {"y": new(N), "z": new(N) if saved else None}
    if case["back"]:
        got.update({"dx": new(case["Kd"])})
        if saved:
            got["dz"] = new(N)
        if act in ("none", "relu"):
            got["dw"] = torch.zeros((case["Kd"], N), dtype=torch.float64, device="cuda")
        if st["bias"] is not None:
            got["db"] = torch.zeros(N, dtype=torch.float64, device="cuda")
    w = st["w"].double()
    wt = w.t().contiguous()
    normal = torch.distributions.Normal(torch.zeros((), dtype=torch.float64, device="cuda"), 1.0)
    for lo in range(0, T, 16384):
        at = slice(lo, lo + 16384)
        x = st["x"][at].double()
        z = x @ w
        if st["bias"] is not None:
            z += st["bias"].double()
        if saved:
            got["z"][at] = z
        y = {"none": z, "relu": z.clamp(min=0), "silu": z * torch.sigmoid(z), "gelu": z * normal.cdf(z)}[act]
        got["y"][at] = y if st["res"] is None else y + st["res"][at].double()
        if case["back"]:
            dz = st["dy"][at].double()
            if act != "none":
                v = st["z"][at].double()
                s = torch.sigmoid(v)
                dz = dz * {"relu": (v > 0).double(), "silu": s + v * s * (1 - s),
                           "gelu": normal.cdf(v) + v * normal.log_prob(v).exp()}[act]
                got["dz"][at] = dz
            got["dx"][at] = dz @ wt
            if "dw" in got:
                got["dw"] += x.t().contiguous() @ dz
            if "db" in got:
                got["db"] += dz.sum(0)
    return got


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    return _exact_few(st) if op == "few" else _exact_norm(st) if op == "norm" else _exact_linear(st)
