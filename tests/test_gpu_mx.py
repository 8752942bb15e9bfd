"""Block-scaled operators on the GPU: 8-bit checkpoints of (a, b) with the backward that reads them, and the
expert products on 4-bit weights, against plain float64 and, where every sum is exact, bit for bit.

Tolerances count roundings: a sum of n products in fp32 is off by at most n * 2^-24 * sum|products| (each
operation rounds by half a step, and the bound holds in any order); one rounding to bf16 by 2^-8 of the value;
the sigmoid (an exponential and a reciprocal of 1 ulp each, an addition, an fp32 argument) by 2^-20 of its value."""
import mx_ref
import numpy as np
import pytest
import torch

from helpers import assert_equal
from routing_permute_groupgemm_amd import _lib, pipeline, synth

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8
W = synth.WORKLOADS


def dev16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits)).view(torch.int16).view(torch.bfloat16).cuda()


def bits(t):
    return pipeline.to_numpy_bits(t)


def normal(shape, seed, std=1.0):
    return synth.operand_bf16(shape, seed, 78, std)


def within(name, got, want, tol):
    got = mx_ref.f64(got) if got.dtype == np.uint16 else got.astype(np.float64)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())}/{bad.size} out of tolerance, first at {i}: got {got[i]!r} "
                             f"want {want[i]!r} tol {tol[i]!r}")


# ---- 8-bit rows -----------------------------------------------------------------------------------------------


def every_pattern():
    """All 65536 bf16 patterns: sorted runs (blocks of one exponent) and shuffled ones (blocks with everything)."""
    a = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    rng = np.random.default_rng(4)
    finite = a[mx_ref.biased_exponent(a) != 255]
    return np.concatenate([a, rng.permutation(a), rng.permutation(finite), finite[:256]]).reshape(-1, 256)


@pytest.mark.parametrize("case", ["patterns", "normal", "one", "zeros"])
def test_pack8_bit_exact(case):
    x = {"patterns": every_pattern, "normal": lambda: normal((777, 448), 1), "one": lambda: normal((1, 64), 2),
         "zeros": lambda: np.array([[0, 0x8000] * 32] * 3, np.uint16)}[case]()
    print(f"[mx] pack8 {case} {x.shape}", flush=True)
    q, s = _lib.moe_pack8(dev16(x))
    v = _lib.moe_unpack8(q, s)
    wq, ws = mx_ref.pack8(x)
    assert_equal("scale", s.cpu().numpy(), ws)
    assert_equal("q", q.cpu().numpy(), wq)
    got, want = mx_ref.f64(bits(v)), mx_ref.unpack8(wq, ws)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("R", [0, 1, 33, 200, 500])
def test_pack8_routed_rows_only(R):
    """Rows behind offsets[e_local] (or behind the buffer, R > rows) are not touched."""
    x = normal((200, 128), 3)
    offsets = torch.tensor([0, R // 2, R], dtype=torch.int32, device="cuda")
    q = torch.full((200, 128), 55, dtype=torch.int8, device="cuda")
    s = torch.full((200, 4), 9, dtype=torch.uint8, device="cuda")
    v = torch.full((200, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    _lib.moe_pack8(dev16(x), q, s, offsets=offsets)
    _lib.moe_unpack8(q, s, v, offsets=offsets)
    n = min(R, 200)
    wq, ws = mx_ref.pack8(x)
    assert_equal("q", q.cpu().numpy()[:n], wq[:n])
    assert_equal("scale", s.cpu().numpy()[:n], ws[:n])
    assert np.array_equal(mx_ref.f64(bits(v))[:n], mx_ref.unpack8(wq, ws)[:n])
    assert (q[n:] == 55).all() and (s[n:] == 9).all() and (v[n:] == 3.0).all()


def test_pack8_past_2_31_elements():
    rows, cols = 524300, 4096  # 2^31 + 49152 values
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    probe = [0, 262143, 524287, 524288, rows - 1]
    x.fill_(1.0)
    want = normal((len(probe), cols), 5)
    x[probe] = dev16(want)
    q, s = _lib.moe_pack8(x)
    v = _lib.moe_unpack8(q, s)
    wq, ws = mx_ref.pack8(want)
    assert_equal("q", q[probe].cpu().numpy(), wq)
    assert_equal("scale", s[probe].cpu().numpy(), ws)
    assert np.array_equal(mx_ref.f64(bits(v[probe])), mx_ref.unpack8(wq, ws))
    assert (v[1:262143] == 1.0).all() and (v[524289:rows - 1] == 1.0).all()


# ---- the gate/up product that saves in 8 bits, and the backward that reads it ---------------------------------

SHAPES = {
    "tiny": W["tiny"].scaled(),
    "ep_share_small": W["ep_share_4k"].scaled(T=512, H=256, F=192),
    "skew_small": W["skew_8k"].scaled(T=1024, H=256, F=128),
    "wide": W["tiny"].scaled(name="wide", T=700, H=192, F=640),
    "one_token": W["tiny"].scaled(name="one_token", T=1, H=64, F=64),
}
TILES = ["auto", "256", "192", "128"]


def routed(shape, seed, cap=None, backward=False, **kw):
    inp = synth.make_inputs(shape, seed=seed, d_out=True)
    dev = pipeline.to_device(inp)
    buf = pipeline.MoeBuffers.allocate(shape, cap=cap, backward=backward, **kw)
    pipeline.route(buf, dev["logits"])
    pipeline.permute(buf, dev["x"])
    torch.cuda.synchronize()
    return inp, dev, buf, min(int(buf.offsets[-1].item()), buf.cap)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("name", list(SHAPES))
def test_save8_equals_packing_the_saved_rows(name, tile, monkeypatch):
    """h is the bf16 call's and (ab8, scale) moe_pack8 of its ab_save, bit for bit, also zero-copy; rows behind
    the routed ones stay."""
    if tile != "auto":
        monkeypatch.setenv("MOE_GEMM_TILE", tile)
    shape = SHAPES[name]
    print(f"[mx] save8 {name} tile={tile}", flush=True)
    inp, dev, buf, R = routed(shape, 21, backward=True)
    _lib.moe_grouped_gemm_swiglu(buf.x_perm, dev["w_gate"], dev["w_up"], buf.offsets, buf.cap, h=buf.h,
                                 ab_save=buf.ab)
    wq, ws = mx_ref.pack8(bits(buf.ab)[:R])
    for zero_copy in (False, True):
        h = torch.full_like(buf.h, 5.0)
        q = torch.full((buf.cap, 2 * shape.F), 55, dtype=torch.int8, device="cuda")
        s = torch.full((buf.cap, shape.F // 16), 9, dtype=torch.uint8, device="cuda")
        if zero_copy:
            _lib.moe_grouped_gemm_swiglu_gather_save8(dev["x"], buf.src, shape.K, dev["w_gate"], dev["w_up"],
                                                      buf.offsets, buf.cap, h=h, ab8=q, ab8_scale=s)
        else:
            _lib.moe_grouped_gemm_swiglu_save8(buf.x_perm, dev["w_gate"], dev["w_up"], buf.offsets, buf.cap, h=h,
                                               ab8=q, ab8_scale=s)
        assert_equal("h", bits(h)[:R], bits(buf.h)[:R])
        assert_equal("scale", s.cpu().numpy()[:R], ws)
        assert_equal("q", q.cpu().numpy()[:R], wq)
        assert (h[R:] == 5.0).all() and (q[R:] == 55).all() and (s[R:] == 9).all()


def test_save8_with_dropped_rows_and_non_finite_tokens():
    shape = SHAPES["ep_share_small"]
    inp, dev, full, R = routed(shape, 22)
    cap = R // 2 + 7
    inp, dev, buf, R = routed(shape, 22, cap=cap, backward=True)
    assert R == cap
    buf.x_perm[3, 5], buf.x_perm[cap - 1, 0] = float("nan"), float("inf")
    _lib.moe_grouped_gemm_swiglu(buf.x_perm, dev["w_gate"], dev["w_up"], buf.offsets, cap, h=buf.h, ab_save=buf.ab)
    h, q, s = _lib.moe_grouped_gemm_swiglu_save8(buf.x_perm, dev["w_gate"], dev["w_up"], buf.offsets, cap)
    wq, ws = mx_ref.pack8(bits(buf.ab))
    assert (ws[3] == 255).all() and (ws[cap - 1] == 255).all() and (ws[4] < 255).all()
    assert_equal("scale", s.cpu().numpy(), ws)
    assert_equal("q", q.cpu().numpy(), wq)
    v = _lib.moe_unpack8(q, s)
    assert torch.isnan(v[3]).all() and torch.isfinite(v[4]).all()


def bwd_reference(dy, w_down, ab, offsets, R):
    """dab, h in float64 and their tolerances, per row of the expert-grouped order."""
    H, F = dy.shape[1], w_down.shape[1]
    dh, mag = np.zeros((R, F)), np.zeros((R, F))
    for j in range(w_down.shape[0]):
        lo, hi = min(offsets[j], R), min(offsets[j + 1], R)
        dh[lo:hi] = dy[lo:hi] @ w_down[j].T
        mag[lo:hi] = np.abs(dy[lo:hi]) @ np.abs(w_down[j].T)
    a, b = ab[:R, :F], ab[:R, F:]
    sg = 1 / (1 + np.exp(-a))
    fa, fb = b * (sg + a * sg * (1 - sg)), a * sg
    # the sum of da's two terms may cancel: its roundings count against their magnitudes
    mag_fa = np.abs(b) * (sg + np.abs(a) * sg * (1 + sg))
    edh = H * U32 * mag
    e = 2.0 ** -18  # a few fp32 operations and the sigmoid
    dab = np.concatenate([dh * fa, dh * fb], 1)
    tol = np.concatenate([edh * np.abs(fa) + e * np.abs(dh) * mag_fa, (edh + e * np.abs(dh)) * np.abs(fb)], 1)
    h = a * sg * b
    return dab, tol + UBF * np.abs(dab) + 1e-37, h, (UBF + e) * np.abs(h) + 1e-37


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("name", list(SHAPES))
def test_bwd8_against_float64(name, tile, monkeypatch):
    if tile != "auto":
        monkeypatch.setenv("MOE_GEMM_TILE", tile)
    shape = SHAPES[name]
    print(f"[mx] bwd8 {name} tile={tile}", flush=True)
    inp, dev, buf, R = routed(shape, 23)
    cap, F = buf.cap, shape.F
    dy, ab = normal((cap, shape.H), 6), normal((cap, 2 * F), 7, 2.0)
    q, s = _lib.moe_pack8(dev16(ab))
    dab = torch.full((cap, 2 * F), 5.0, dtype=torch.bfloat16, device="cuda")
    h = torch.full((cap, F), 5.0, dtype=torch.bfloat16, device="cuda")
    _lib.moe_grouped_gemm_swiglu_bwd8(dev16(dy), dev["w_down"], buf.offsets, cap, q, s, dab=dab, h=h)
    wd, tol, wh, htol = bwd_reference(mx_ref.f64(dy), mx_ref.f64(inp["w_down"]), mx_ref.unpack8(*mx_ref.pack8(ab)),
                                      bits(buf.offsets), R)
    within("dab", bits(dab)[:R], wd, tol)
    within("h", bits(h)[:R], wh, htol)
    assert (dab[R:] == 5.0).all() and (h[R:] == 5.0).all()
    # without h, the same dab
    again, none = _lib.moe_grouped_gemm_swiglu_bwd8(dev16(dy), dev["w_down"], buf.offsets, cap, q, s, want_h=False)
    assert none is None
    assert_equal("dab without h", bits(again)[:R], bits(dab)[:R])


def test_bwd8_equals_the_bf16_backward_on_the_same_values(monkeypatch):
    """With ab the bf16 values that the blocks hold, the bf16 epilogue's dab in the 256-row body (the same
    arithmetic on the same values; the smaller bodies of the bf16 epilogue multiply in another order)."""
    monkeypatch.setenv("MOE_GEMM_TILE", "256")
    shape = W["fwdbwd_16k"].scaled(name="wide256", T=2048, H=128, F=256, E=4, K=2)
    inp, dev, buf, R = routed(shape, 24)
    ab = normal((buf.cap, 2 * shape.F), 8, 2.0)
    dy = dev16(normal((buf.cap, shape.H), 9))
    q, s = _lib.moe_pack8(dev16(ab))
    v = _lib.moe_unpack8(q, s)
    dab8, h8 = _lib.moe_grouped_gemm_swiglu_bwd8(dy, dev["w_down"], buf.offsets, buf.cap, q, s)
    dab = torch.empty_like(dab8)
    _lib.moe_grouped_gemm(dy, dev["w_down"], None, 1, buf.offsets, shape.H, shape.F, buf.cap, dab,
                          epilogue=_lib.MOE_EPI_SWIGLU_BWD, ab=v)
    assert_equal("dab", bits(dab8)[:R], bits(dab)[:R])


def test_bwd8_is_the_gradient_by_differences():
    """<dab, v> against central differences of sum dh * silu(a) b in the direction v, in float64.  dh = dy . Wd^T
    is exact (small integers); the difference quotient's own error is O(eps^2)."""
    shape = W["tiny"].scaled(name="fd", T=96, H=64, F=64, E=3, K=1)
    rng = np.random.default_rng(10)
    inp, dev, buf, R = routed(shape, 25)
    cap, F = buf.cap, shape.F
    dy = synth.f32_to_bf16_bits(rng.integers(-2, 3, (cap, 64)).astype(np.float32))
    wd = synth.f32_to_bf16_bits(rng.integers(-2, 3, (3, F, 64)).astype(np.float32))
    ab = normal((cap, 2 * F), 11, 1.5)
    q, s = _lib.moe_pack8(dev16(ab))
    dab, _ = _lib.moe_grouped_gemm_swiglu_bwd8(dev16(dy), dev16(wd), buf.offsets, cap, q, s)
    off = bits(buf.offsets)
    dh = np.zeros((cap, F))
    for j in range(3):
        dh[off[j]:off[j + 1]] = mx_ref.f64(dy)[off[j]:off[j + 1]] @ mx_ref.f64(wd)[j].T
    x = mx_ref.unpack8(*mx_ref.pack8(ab))

    def loss(z):
        a, b = z[:, :F], z[:, F:]
        return dh * a / (1 + np.exp(-a)) * b

    got, eps = mx_ref.f64(bits(dab)), 1e-5
    for half in (0, 1):
        v = np.zeros_like(x)
        v[:, half * F:(half + 1) * F] = 1.0
        want = (loss(x + eps * v) - loss(x - eps * v)) / (2 * eps)
        a, b = np.abs(x[:, :F]), np.abs(x[:, F:])
        # bf16 rounding, 2^-18 of the terms, and eps^2 |third derivative| (below 4 (1 + |a|) (1 + |b|) |dh|) plus
        # the quotient's rounding, 2^-52 |loss| / eps
        tol = UBF * np.abs(want) + (2.0 ** -17) * np.abs(dh) * (1 + a) * (1 + b) + 1e-30
        within("da db"[3 * half:3 * half + 2], got[:R, half * F:(half + 1) * F], want[:R], tol[:R])


# ---- 4-bit weights --------------------------------------------------------------------------------------------


@pytest.mark.parametrize("E,Kd,N", [(1, 64, 64), (2, 128, 192), (3, 192, 64), (5, 448, 128), (1, 1024, 320)])
def test_pack4_bit_exact(E, Kd, N):
    print(f"[mx] pack4 {E} {Kd} {N}", flush=True)
    w = normal((E, Kd, N), 12, 0.02)
    flat = w.reshape(-1)
    flat[:128] = every_pattern()[200, :128]          # large and tiny magnitudes
    w[0, 32, 3], w[E - 1, Kd - 1, N - 1], w[0, 5, 1] = 0x7FC0, 0xFF80, 0x0001  # NaN, -inf, the smallest denormal
    w[E - 1, Kd - 64:Kd - 32, 7] = 0                   # a block of zeros
    codes, s = mx_ref.codes4(w)
    wq, ws = mx_ref.layout4(codes, s)
    q4, s4 = _lib.moe_pack4(dev16(w))
    live = np.zeros_like(ws, bool)
    for kb in range(Kd // 32):
        live[:, :, kb // 4, 16 * (kb % 4):16 * (kb % 4) + 16] = True
    assert_equal("q4", q4.cpu().numpy(), wq)
    assert_equal("s4", np.where(live, s4.cpu().numpy(), 0), ws)
    assert (s4.cpu().numpy()[~live] < 255).all()       # the codes behind Kd stand for 0
    v = _lib.moe_unpack4(q4, s4, Kd)
    assert np.array_equal(mx_ref.f64(bits(v)), mx_ref.values4(codes, s), equal_nan=True)


def test_pack4_every_scale():
    """A block per exponent of the largest magnitude, every mantissa below it."""
    w = np.zeros((1, 64, 256), np.uint16)
    for e in range(256):
        m = np.minimum(np.arange(32) * 4 + (e << 7), (e << 7) + 127)
        w[0, :32, e] = m
        w[0, 32:, e] = 0x8000 | np.maximum(m - 128 * np.arange(32), 0)
    codes, s = mx_ref.codes4(w)
    q4, s4 = _lib.moe_pack4(dev16(w))
    wq, _ = mx_ref.layout4(codes, s)
    assert_equal("q4", q4.cpu().numpy(), wq)
    assert np.array_equal(mx_ref.f64(bits(_lib.moe_unpack4(q4, s4, 64))), mx_ref.values4(codes, s), equal_nan=True)


def plan4(counts, seed, T, K):
    """Rows per expert -> (offsets, src with distinct random pairs) on the GPU and as numpy."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = np.random.default_rng(seed).permutation(T * K)[:off[-1]].astype(np.int32)
    return off, src


def reference4(x, w, off):
    """Per-row product in float64 and its tolerance before the last rounding."""
    R, N = off[-1], w.shape[2]
    y, tol = np.zeros((R, N)), np.zeros((R, N))
    for j in range(w.shape[0]):
        lo, hi = off[j], off[j + 1]
        y[lo:hi] = x[lo:hi] @ w[j]
        tol[lo:hi] = x.shape[1] * U32 * (np.abs(x[lo:hi]) @ np.abs(w[j]))
    return y, tol


COUNTS = {
    "wide_rows": [20] * 20,
    "even": [13, 9, 11, 14] * 6,
    "tens": [25, 60, 31, 40, 33, 28] * 2,
    "one_row": [1],
    "single_token": [0, 1, 0, 0, 1, 0, 1, 1],
    "ragged": [3, 0, 17, 16, 1, 33, 0, 15],
    "none": [0, 0, 0],
    "many": [70, 129, 0, 64, 200],
    "last_only": [0] * 130 + [5],
    "hundred": [(5 * i) % 3 for i in range(100)],
    "wide": [(7 * i) % 4 for i in range(300)],
    "most_experts": [(i % 9 == 4) * 2 for i in range(512)],
}


def check_combined(got, pos, gates, y, ey):
    """sum_k gate * y over the present pairs: K roundings on top of the rows' own, and the last one to bf16."""
    T, K = pos.shape
    out, tol = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for k in range(K):
        ok = pos[:, k] >= 0
        g = gates[ok, k, None].astype(np.float64)
        out[ok] += g * y[pos[ok, k]]
        tol[ok] += g * (ey[pos[ok, k]] + 2 * K * U32 * np.abs(y[pos[ok, k]]))
    within("out", got, out, tol + UBF * np.abs(out) + 1e-37)


@pytest.mark.parametrize("H,F", [(64, 64), (128, 192), (192, 128), (320, 64), (1408, 320), (2112, 1984)])
@pytest.mark.parametrize("counts", list(COUNTS))
def test_gemm4_against_float64(counts, H, F):
    n = COUNTS[counts]
    if len(n) >= 100 and H * F > 128 * 192:
        H, F = 64, 128
    if H * F > 1408 * 320 and counts not in ("wide_rows", "even", "tens"):
        H, F = 64, 1088
    K, R = 4, sum(n)
    T = max(R, 8)
    print(f"[mx] gemm4 {counts} H={H} F={F} R={R}", flush=True)
    off, src = plan4(n, 30, T, K)
    cap = R + 3
    x = normal((T, H), 31)
    mats = {m: normal((len(n), *s), 32 + i, 0.05) for i, (m, s) in
            enumerate((("gate", (H, F)), ("up", (H, F)), ("down", (F, H))))}
    packed = {m: _lib.moe_pack4(dev16(w)) for m, w in mats.items()}
    vals = {m: mx_ref.values4(*mx_ref.codes4(w)) for m, w in mats.items()}
    offsets = torch.from_numpy(off).cuda()
    srcd = torch.from_numpy(np.concatenate([src, np.full(3, -1, np.int32)])).cuda()
    h = torch.full((cap, F), 5.0, dtype=torch.bfloat16, device="cuda")
    _lib.moe_grouped_gemm4_swiglu(dev16(x), srcd, K, packed["gate"], packed["up"], offsets, cap, h=h)
    xr = mx_ref.f64(x)[src // K]
    a, ea = reference4(xr, vals["gate"], off)
    b, eb = reference4(xr, vals["up"], off)
    sg = 1 / (1 + np.exp(-a))
    want = a * sg * b
    # |d silu| <= 1.1
    tol = 1.1 * ea * np.abs(b) + np.abs(a * sg) * eb + 1.1 * ea * eb + (UBF + 2.0 ** -18) * np.abs(want) + 1e-37
    within("h", bits(h)[:R], want, tol)
    assert (h[R:] == 5.0).all()
    # rows already in expert order, and a second run: the same bits
    xp = torch.full((cap, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    xp[:R] = dev16(x[src // K]) if R else xp[:0]
    h2 = torch.full((cap, F), 5.0, dtype=torch.bfloat16, device="cuda")
    _lib.moe_grouped_gemm4_swiglu(xp, None, None, packed["gate"], packed["up"], offsets, cap, h=h2)
    assert_equal("h from ordered rows", bits(h2), bits(h))
    # down, on rows whose tail is NaN
    hin = torch.full((cap, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    hin[:R] = h[:R]
    y = torch.full((cap, H), 5.0, dtype=torch.bfloat16, device="cuda")
    _lib.moe_grouped_gemm4(hin, packed["down"], offsets, cap, c=y)
    wy, ey = reference4(mx_ref.f64(bits(h))[:R], vals["down"], off)
    within("y", bits(y)[:R], wy, ey + UBF * np.abs(wy) + 1e-37)
    assert (y[R:] == 5.0).all()
    # down and combine in one: y, and the gated sum of the unrounded rows (absent pairs -1)
    pos = np.full(T * K, -1, np.int32)
    pos[src] = np.arange(R)
    gates = np.random.default_rng(37).random((T, K)).astype(np.float32)
    y2 = torch.full((cap, H), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (hin, packed["down"], offsets, cap, torch.from_numpy(pos.reshape(T, K)).cuda(), torch.from_numpy(gates).cuda())
    out = _lib.moe_grouped_gemm4_combine(*args, y=y2)
    within("y of the combined call", bits(y2)[:R], wy, ey + UBF * np.abs(wy) + 1e-37)
    assert (y2[R:] == 5.0).all()
    check_combined(bits(out), pos.reshape(T, K), gates, wy, ey)
    assert_equal("without y", bits(_lib.moe_grouped_gemm4_combine(*args)), bits(out))


@pytest.mark.parametrize("rows,Kd,N", [(1, 4096, 2112), (3, 4096, 2112), (9, 4096, 2112), (20, 4096, 2112),
                                       (28, 4096, 2112), (40, 4096, 2112), (9, 1024, 6464), (40, 1024, 6464),
                                       (5, 192, 6464), (20, 192, 6464)])
def test_gemm4_large_matrices(rows, Kd, N):
    """Matrices past half the last-level cache (non-temporal loads for the experts of one row tile) at every row
    tile, and many columns (256 a workgroup, the last of them partly empty), of small matrices too: 40 experts of
    about `rows` rows, one of them with three times as many (18 for one row) and one with none, against float64 on
    the GPU."""
    E = 40
    rng = np.random.default_rng(rows)
    n = rng.integers(max(rows - 3, 1), rows + 2, E)
    n[7], n[11] = 3 * rows if rows > 1 else 18, 0
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    R = int(off[-1])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    mats = [(torch.randn((E, Kd, N), generator=gen, device="cuda") * 0.02).to(torch.bfloat16) for _ in range(2)]
    x = torch.randn((R, Kd), generator=gen, device="cuda").to(torch.bfloat16)
    packed = [_lib.moe_pack4(m) for m in mats]
    offsets = torch.from_numpy(off).cuda()
    print(f"[mx] gemm4 large, {R} rows", flush=True)
    c = _lib.moe_grouped_gemm4(x, packed[0], offsets, R)
    h = _lib.moe_grouped_gemm4_swiglu(x, None, None, packed[0], packed[1], offsets, R)
    vals = [_lib.moe_unpack4(*p, Kd) for p in packed]
    for j in range(E):
        lo, hi = off[j], off[j + 1]
        xr = x[lo:hi].double()
        a, b = (xr @ v[j].double() for v in vals)
        ea, eb = (Kd * U32 * (xr.abs() @ v[j].double().abs()) for v in vals)
        assert ((c[lo:hi].double() - a).abs() <= ea + UBF * a.abs()).all(), j
        sg = torch.sigmoid(a)
        want = a * sg * b
        tol = 1.1 * ea * b.abs() + (a * sg).abs() * eb + 1.1 * ea * eb + (UBF + 2.0 ** -18) * want.abs() + 1e-37
        assert ((h[lo:hi].double() - want).abs() <= tol).all(), j


@pytest.mark.parametrize("counts", ["ragged", "many"])
def test_gemm4_exact_on_integers(counts):
    """Small integers in every operand: fp32 sums are exact in any order, so the bf16 results are too."""
    n = COUNTS[counts]
    Kd, N, R = 448, 128, sum(COUNTS[counts])
    rng = np.random.default_rng(33)
    a = rng.integers(-8, 9, (R, Kd)).astype(np.float32)
    w = np.array([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], np.float32)[rng.integers(0, 11, (len(n), Kd, N))]
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    y = _lib.moe_grouped_gemm4(dev16(synth.f32_to_bf16_bits(a)), _lib.moe_pack4(dev16(synth.f32_to_bf16_bits(w))),
                               torch.from_numpy(off).cuda(), R)
    want, _ = reference4(a.astype(np.float64), w.astype(np.float64), off)
    assert np.abs(want).max() < 2 ** 24
    assert_equal("y", bits(y), synth.f32_to_bf16_bits(want.astype(np.float32)))


def test_gemm4_bad_indices_non_finite_and_dropped_rows():
    H, F, K, T = 128, 64, 2, 5
    x, w = normal((T, H), 34), normal((2, H, F), 35, 0.05)
    w[1, 40, 9] = 0x7F80                                  # an infinity in a block of expert 1
    x[4, 7] = 0x7FC0                                      # a NaN in token 4
    g, u = _lib.moe_pack4(dev16(w)), _lib.moe_pack4(dev16(normal((2, H, F), 36, 0.05)))
    offsets = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    src = torch.tensor([0, 99, -7, 8, 2, 4, 6, 1, 3], dtype=torch.int32, device="cuda")  # 8 -> token 4
    h = _lib.moe_grouped_gemm4_swiglu(dev16(x), src, K, g, u, offsets, 9)
    assert (h[1:3] == 0).all() and torch.isnan(h[3]).all()   # outside [0, T*K): a zero row
    assert torch.isfinite(h[0]).all() and torch.isnan(h[4:9, 9]).all()
    assert torch.isfinite(h[4:9, :9]).all() and torch.isfinite(h[4:9, 10:]).all()
    # capacity below the routed rows: the rest is dropped
    c = torch.full((9, F), 5.0, dtype=torch.bfloat16, device="cuda")
    _lib.moe_grouped_gemm4_swiglu(dev16(x), src, K, g, u, offsets, 6, h=c)
    assert_equal("kept rows", bits(c)[:6], bits(h)[:6])
    assert (c[6:] == 5.0).all()


def test_binding_refuses_wrong_shapes():
    dev = "cuda"
    q4, s4 = _lib.moe_pack4(torch.zeros((2, 192, 64), dtype=torch.bfloat16, device=dev))
    offsets = torch.zeros(3, dtype=torch.int32, device=dev)
    a = torch.zeros((4, 192), dtype=torch.bfloat16, device=dev)
    src = torch.zeros(4, dtype=torch.int32, device=dev)
    for call in (
        lambda: _lib.moe_grouped_gemm4(a[:, :64].contiguous(), (q4, s4), offsets, 4),     # contraction differs
        lambda: _lib.moe_grouped_gemm4(a, (q4, s4), offsets[:2], 4),                      # offsets too short
        lambda: _lib.moe_grouped_gemm4(a, (q4, s4), offsets, 5),                          # more rows than a has
        lambda: _lib.moe_grouped_gemm4(a, (q4, s4[:1]), offsets, 4),
        lambda: _lib.moe_grouped_gemm4(a.t(), (q4, s4), offsets, 4),
        lambda: _lib.moe_grouped_gemm4_swiglu(a, src[:3], 1, (q4, s4), (q4, s4), offsets, 4),
        lambda: _lib.moe_grouped_gemm4_swiglu(a, src, 1, (q4, s4), (q4[:1], s4[:1]), offsets, 4),
        lambda: _lib.moe_grouped_gemm4_swiglu(a, src, 0, (q4, s4), (q4, s4), offsets, 4),
        lambda: _lib.moe_grouped_gemm4_swiglu(a, src, 1, (q4, s4), (q4, s4), offsets, 4, h=a),
        lambda: _lib.moe_pack4(torch.zeros((2, 96, 64), dtype=torch.bfloat16, device=dev)),
        lambda: _lib.moe_unpack4(q4, s4, 128),
        lambda: _lib.moe_pack8(torch.zeros((2, 96), dtype=torch.bfloat16, device=dev)),
        lambda: _lib.moe_pack8(a, q=torch.zeros((4, 64), dtype=torch.int8, device=dev)),
        lambda: _lib.moe_unpack8(torch.zeros((4, 64), dtype=torch.int8, device=dev), s4),
        lambda: _lib.moe_pack8(a, offsets=offsets.long()),
    ):
        with pytest.raises(_lib.MoeError):
            call()


def test_nothing_to_do():
    """No expert, no row, no token: nothing is written, and the combined sum of no rows is 0."""
    dev = "cuda"
    q4, s4 = _lib.moe_pack4(torch.zeros((0, 64, 64), dtype=torch.bfloat16, device=dev))
    assert q4.shape == (0, 4, 1, 64, 16) and s4.shape == (0, 4, 1, 64)
    offsets = torch.zeros(1, dtype=torch.int32, device=dev)
    x = torch.ones((5, 64), dtype=torch.bfloat16, device=dev)
    src = torch.zeros(3, dtype=torch.int32, device=dev)
    h = torch.full((3, 64), 5.0, dtype=torch.bfloat16, device=dev)
    _lib.moe_grouped_gemm4_swiglu(x, src, 1, (q4, s4), (q4, s4), offsets, 3, h=h)
    _lib.moe_grouped_gemm4(x, (q4, s4), offsets, 3, c=h)
    assert (h == 5.0).all()
    w = _lib.moe_pack4(torch.ones((2, 64, 64), dtype=torch.bfloat16, device=dev))
    off2 = torch.tensor([0, 0, 0], dtype=torch.int32, device=dev)
    for weights, off, cap in (((q4, s4), offsets, 3), (w, off2, 3), (w, off2, 0)):
        out = torch.full((5, 64), 5.0, dtype=torch.bfloat16, device=dev)
        _lib.moe_grouped_gemm4_combine(x, weights, off, cap, torch.full((5, 2), -1, dtype=torch.int32, device=dev),
                                       torch.ones((5, 2), device=dev), out=out)
        assert (out == 0).all()
    assert _lib.moe_grouped_gemm4(x, w, off2, 0).shape == (0, 64)
    q, s = _lib.moe_pack8(torch.zeros((0, 64), dtype=torch.bfloat16, device=dev))
    assert _lib.moe_unpack8(q, s).shape == (0, 64)
    wb = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device=dev)
    assert _lib.moe_grouped_gemm_swiglu_save8(x, wb, wb, off2, 0)[1].shape == (0, 128)
    assert _lib.moe_grouped_gemm_swiglu_bwd8(x, wb, off2, 0, q.new_empty((0, 128)), s.new_empty((0, 4)))[0].shape == (0, 128)


def test_buffers_past_2_31_elements():
    """262 300 rows: the 8192 bytes of a row's (a, b) and the fp32 and bf16 rows of the products lie on both sides of
    2 and 4 GiB.  Rows there equal those of a call on them alone (h and the bytes bit for bit, the rest within its
    tolerance against float64)."""
    rows, H, F = 262300, 64, 4096
    gen = torch.Generator(device="cuda")
    gen.manual_seed(50)
    x = torch.randn((rows, H), generator=gen, device="cuda").to(torch.bfloat16)
    w = [(torch.randn((1, H, F), generator=gen, device="cuda") * 0.1).to(torch.bfloat16) for _ in range(2)]
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 131071, 131072, 262143, 262144, 262145, rows - 1], device="cuda")
    few = torch.tensor([0, at.numel()], dtype=torch.int32, device="cuda")
    print("[mx] large save8", flush=True)
    h, q, s = _lib.moe_grouped_gemm_swiglu_save8(x, w[0], w[1], offsets, rows)
    h1, q1, s1 = _lib.moe_grouped_gemm_swiglu_save8(x[at], w[0], w[1], few, at.numel())
    for a, b in ((h, h1), (q, q1), (s, s1)):
        assert torch.equal(a[at], b)
    assert torch.equal(_lib.moe_unpack8(q, s)[at], _lib.moe_unpack8(q1, s1))
    print("[mx] large bwd8", flush=True)
    wd = (torch.randn((1, F, H), generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    dab, h = _lib.moe_grouped_gemm_swiglu_bwd8(x, wd, offsets, rows, q, s)
    wdab, tol, wh, htol = bwd_reference(mx_ref.f64(bits(x[at])), mx_ref.f64(bits(wd)),
                                        mx_ref.f64(bits(_lib.moe_unpack8(q1, s1))), bits(few), at.numel())
    within("dab", bits(dab[at]), wdab, tol)
    within("h", bits(h[at]), wh, htol)
    del dab, q, s
    print("[mx] large 4-bit", flush=True)
    packed = [_lib.moe_pack4(m) for m in w]
    vals = [mx_ref.f64(bits(_lib.moe_unpack4(*p, H)))[0] for p in packed]
    xr = mx_ref.f64(bits(x[at]))
    c = _lib.moe_grouped_gemm4(torch.cat((x, x)), packed[0], 2 * offsets, 2 * rows)
    for half in (0, rows):
        want, mag = xr @ vals[0], np.abs(xr) @ np.abs(vals[0])
        within("c", bits(c[at + half]), want, H * U32 * mag + UBF * np.abs(want) + 1e-37)
    del c
    pos = torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).reshape(-1, 2).contiguous()
    gates = torch.rand(pos.shape, generator=gen, device="cuda")
    out = _lib.moe_grouped_gemm4_combine(x, packed[0], offsets, rows, pos, gates)
    t = [0, 1, 65535, 65536, 131149]
    for i in t:
        g, p = bits(gates)[i].astype(np.float64), bits(pos)[i]
        xr = mx_ref.f64(bits(x[torch.from_numpy(p).cuda().long()]))
        r = xr @ vals[0]
        mag = H * U32 * (np.abs(xr) @ np.abs(vals[0])) + 4 * U32 * np.abs(r)
        want = (g[:, None] * r).sum(0)
        within("out", bits(out[i]), want, (g[:, None] * mag).sum(0) + UBF * np.abs(want) + 1e-37)


def test_two_streams_at_once():
    """The same calls on two streams with buffers of their own: each gives the bits that it gives alone."""
    shape = SHAPES["ep_share_small"]
    inp, dev, buf, R = routed(shape, 26, backward=True)
    ab = dev16(normal((buf.cap, 2 * shape.F), 51, 2.0))
    packed = {k: _lib.moe_pack4(dev[k]) for k in ("w_gate", "w_up", "w_down")}

    def chain():
        h, q, s = _lib.moe_grouped_gemm_swiglu_save8(buf.x_perm, dev["w_gate"], dev["w_up"], buf.offsets, buf.cap)
        dab, h2 = _lib.moe_grouped_gemm_swiglu_bwd8(buf.x_perm, dev["w_down"], buf.offsets, buf.cap, q, s)
        h4 = _lib.moe_grouped_gemm4_swiglu(dev["x"], buf.src, shape.K, packed["w_gate"], packed["w_up"], buf.offsets,
                                           buf.cap)
        out = _lib.moe_grouped_gemm4_combine(h4, packed["w_down"], buf.offsets, buf.cap, buf.pos, buf.gates)
        p, ps = _lib.moe_pack8(ab)
        return [h[:R], q[:R], s[:R], dab[:R], h2[:R], h4[:R], out, p, ps]

    want = [t.clone() for t in chain()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(chain())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    # and by argument instead of the current stream
    q, s = _lib.moe_pack8(ab, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(q, want[7]) and torch.equal(s, want[8])


# ---- together, as the pipeline runs them ----------------------------------------------------------------------


@pytest.mark.parametrize("zero_copy", [False, True])
@pytest.mark.parametrize("name", ["tiny", "ep_share_small", "skew_small"])
def test_training_step_with_8bit_checkpoint(name, zero_copy):
    """The forward's output is the plain step's bit for bit.  The backward's dab and h are the SwiGLU's derivative
    and value at the saved values; what follows (dX, dW) is the bf16 calls on them."""
    shape = SHAPES[name].scaled(backward=True)
    inp = synth.make_inputs(shape, seed=40, d_out=True)
    dev = pipeline.to_device(inp)
    ref = pipeline.MoeBuffers.allocate(shape, zero_copy=zero_copy)
    buf = pipeline.MoeBuffers.allocate(shape, zero_copy=zero_copy, checkpoint8=True)
    assert buf.ab is None and ref.ab8 is None
    pipeline.forward(ref, dev)
    pipeline.forward(buf, dev)
    assert_equal("out", bits(buf.out), bits(ref.out))
    R = min(int(buf.offsets[-1].item()), buf.cap)
    buf.h.fill_(float("nan"))  # not kept between forward and backward
    pipeline.backward(ref, dev)
    pipeline.backward(buf, dev)
    # the same backward in bf16 from the unpacked (a, b): identical from there on
    ref.ab.copy_(_lib.moe_unpack8(buf.ab8, buf.ab8_scale))
    wd, tol, wh, htol = bwd_reference(mx_ref.f64(bits(buf.dy_perm))[:R], mx_ref.f64(inp["w_down"]),
                                      mx_ref.f64(bits(ref.ab))[:R], bits(buf.offsets), R)
    within("dab", bits(buf.dab)[:R], wd, tol)
    within("h", bits(buf.h)[:R], wh, htol)
    dx = _lib.moe_grouped_gemm(buf.dab, dev["w_gate"], dev["w_up"], 1, buf.offsets, shape.F, shape.H, buf.cap,
                               torch.empty_like(ref.dx_perm))
    assert_equal("dx", bits(buf.dx), bits(_lib.moe_combine(dx, buf.pos, None)))
    dw = _lib.moe_wgrad(buf.h, shape.F, buf.dy_perm, shape.H, buf.offsets, shape.EL, shape.F, shape.H, buf.cap)
    assert_equal("dw_down", bits(buf.dw_down), bits(dw))
    # against the bf16 checkpoint: the 8-bit rounding of (a, b) is at most 1/128 of a block's largest value
    for n in ("dx", "dw_gate", "dw_up", "dw_down"):
        got, want = getattr(buf, n).double(), getattr(ref, n).double()
        assert (got - want).norm() <= 0.03 * want.norm(), n
    assert_equal("dlogits", bits(buf.dlogits), bits(ref.dlogits))


@pytest.mark.parametrize("T", [1, 2, 37, 300])
@pytest.mark.parametrize("name", ["tiny", "ep_share_small", "skew_small"])
def test_decode_step_on_4bit_weights(name, T):
    """forward4 from routing to output; the routing is the bf16 forward's."""
    shape = SHAPES[name].scaled(T=T)
    inp = synth.make_inputs(shape, seed=41)
    dev = pipeline.to_device(inp)
    dev.update(pipeline.pack_weights4(dev))
    ref = pipeline.MoeBuffers.allocate(shape, zero_copy=True, backward=False)
    buf = pipeline.MoeBuffers.allocate(shape, weights4=True)
    assert buf.y is None and buf.zero_copy
    pipeline.forward4(buf, dev)
    pipeline.forward(ref, dev)
    assert_equal("routing", bits(buf.pos), bits(ref.pos))
    R = min(int(buf.offsets[-1].item()), buf.cap)
    h, off = mx_ref.f64(bits(buf.h)[:R]), np.minimum(bits(buf.offsets), R)
    w = {k: mx_ref.f64(bits(_lib.moe_unpack4(*dev[k + "4"], kd)))
         for k, kd in (("w_gate", shape.H), ("w_up", shape.H), ("w_down", shape.F))}
    xr = mx_ref.f64(inp["x"])[bits(buf.src)[:R] // shape.K]
    a, ea = reference4(xr, w["w_gate"], off)
    b, eb = reference4(xr, w["w_up"], off)
    sg = 1 / (1 + np.exp(-a))
    within("h", h, a * sg * b, 1.1 * ea * np.abs(b) + np.abs(a * sg) * eb + 1.1 * ea * eb
           + (UBF + 2.0 ** -18) * np.abs(a * sg * b) + 1e-37)
    y, ey = reference4(h, w["w_down"], off)
    check_combined(bits(buf.out), bits(buf.pos), bits(buf.gates), y, ey)
    with pytest.raises(_lib.MoeError):
        pipeline.forward4(ref, dev)
    with pytest.raises(_lib.MoeError):
        pipeline.forward(buf, dev)


def test_replay_from_a_graph_and_another_stream():
    """Both paths captured together; every replay reproduces the eager bits after the outputs are clobbered."""
    shape = SHAPES["ep_share_small"].scaled(backward=True)
    inp = synth.make_inputs(shape, seed=42, d_out=True)
    dev = pipeline.to_device(inp)
    dev.update(pipeline.pack_weights4(dev))
    train = pipeline.MoeBuffers.allocate(shape, checkpoint8=True)
    serve = pipeline.MoeBuffers.allocate(shape.scaled(backward=False), weights4=True)

    def step():
        pipeline.forward(train, dev)
        pipeline.backward(train, dev)
        pipeline.forward4(serve, dev)

    outs = [train.out, train.dx, train.dw_gate, train.dw_up, train.dw_down, train.dlogits, serve.out]
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in outs:
        t.fill_(7)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in outs + [train.h, serve.h, serve.ws4]:
            t.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
