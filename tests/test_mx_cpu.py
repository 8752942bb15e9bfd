"""Block-scaled storage on the CPU: the reference's own properties, and the entry points' refusals."""
import mx_ref
import numpy as np
import pytest
import torch

from routing_permute_groupgemm_amd import _lib, synth

FAKE, MIS = 0x10000, 0x10004  # never dereferenced: validation fails first


def normal_bits(shape, seed, std=1.0):
    return synth.operand_bf16(shape, seed, 77, std)


@pytest.mark.parametrize("std", [1e-30, 1.0, 1e30])
def test_8bit_error_is_at_most_half_a_step(std):
    bits = normal_bits((64, 256), 1, std)
    q, s = mx_ref.pack8(bits)
    x, v = mx_ref.f64(bits), mx_ref.unpack8(q, s)
    half = np.repeat(np.ldexp(1.0, s.astype(int) - 134), 32, axis=1)
    assert (np.abs(v - x) <= half).all()
    m = np.repeat(np.abs(x).reshape(64, -1, 32).max(2), 32, axis=1)
    assert (half <= m / 128).all()
    # a value is a bf16: it survives the rounding
    f = v.astype(np.float32)
    assert np.array_equal(synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(f)), f)


def test_8bit_largest_mantissa_is_clamped_within_half_a_step():
    bits = np.zeros((1, 64), np.uint16)
    bits[0, 0], bits[0, 33] = 0x3FFF, 0xFF7F  # 1.9921875; the largest negative finite value
    q, s = mx_ref.pack8(bits)
    assert q[0, 0] == 127 and s[0, 0] == 127 and q[0, 33] == -127 and s[0, 1] == 254
    assert abs(mx_ref.unpack8(q, s)[0, 0] - 1.9921875) == 2.0 ** (127 - 134)


def test_4bit_error_and_repacking():
    bits = normal_bits((2, 128, 64), 2, 0.02)
    c, s = mx_ref.codes4(bits)
    x, v = mx_ref.f64(bits), mx_ref.values4(c, s)
    unit = np.repeat(np.ldexp(1.0, s - 127), 32, axis=1)
    u, err = np.abs(x) / unit, np.abs(v - x) / unit
    assert (u < 8).all()
    # half a gap below 2, 4 and 6, and what is cut off above 6
    bound = np.where(u <= 2, 0.25, np.where(u <= 4, 0.5, np.where(u <= 6, 1.0, u - 6)))
    assert (err <= bound).all()
    # the values pack to themselves, whatever scale their block had
    for shift in (0, 1, 2):
        c2 = np.where((c & 7) >= 2 + 2 * shift, 0, c)  # smaller codes only: a block with a scale larger than needed
        w = mx_ref.values4(c2, s)
        again = mx_ref.values4(*mx_ref.codes4(synth.f32_to_bf16_bits(w.astype(np.float32))))
        assert np.array_equal(again, w)
    w = mx_ref.values4(c, s)
    assert np.array_equal(mx_ref.values4(*mx_ref.codes4(synth.f32_to_bf16_bits(w.astype(np.float32)))), w)


def test_layout4_holds_every_code_once():
    rng = np.random.default_rng(3)
    c = rng.integers(0, 16, (1, 192, 64)).astype(np.uint8)
    q4, s4 = mx_ref.layout4(c, np.full((1, 6, 64), 120))
    flat = np.concatenate([(q4 & 15).ravel(), (q4 >> 4).ravel()])
    got = np.bincount(flat, minlength=16)
    want = np.bincount(c.ravel(), minlength=16)
    want[0] += flat.size - c.size  # behind Kd
    assert np.array_equal(got, want)


def test_pack8_refusals():
    lib = _lib.load()
    p, u = lib.moe_pack8, lib.moe_unpack8
    assert p(FAKE, 4, 96, None, 0, FAKE, FAKE, None) == -2
    assert p(FAKE, -1, 64, None, 0, FAKE, FAKE, None) == -1
    assert p(FAKE, 1 << 31, 64, None, 0, FAKE, FAKE, None) == -1
    assert p(FAKE, 4, 64, FAKE, 513, FAKE, FAKE, None) == -1
    assert p(None, 4, 64, None, 0, FAKE, FAKE, None) == -1
    assert p(FAKE, 4, 64, None, 0, FAKE, None, None) == -1
    assert p(MIS, 4, 64, None, 0, FAKE, FAKE, None) == -3
    assert p(None, 0, 64, None, 0, None, None, None) == 0
    assert u(FAKE, FAKE, 4, 32, None, 0, FAKE, None) == -2
    assert u(FAKE, None, 4, 64, None, 0, FAKE, None) == -1
    assert u(FAKE, FAKE, 4, 64, MIS, 2, FAKE, None) == -3
    assert u(None, None, 4, 0, None, 0, None, None) == 0


def test_pack4_refusals():
    lib = _lib.load()
    p, u = lib.moe_pack4, lib.moe_unpack4
    assert p(FAKE, 2, 96, 64, FAKE, FAKE, None) == -2
    assert p(FAKE, 2, 64, 32, FAKE, FAKE, None) == -2
    assert p(FAKE, 513, 64, 64, FAKE, FAKE, None) == -1
    assert p(FAKE, -1, 64, 64, FAKE, FAKE, None) == -1
    assert p(FAKE, 1, 65536, 16384, FAKE, FAKE, None) == -1  # 2 GiB of bf16 in one expert
    assert p(None, 2, 64, 64, FAKE, FAKE, None) == -1
    assert p(FAKE, 2, 64, 64, MIS, FAKE, None) == -3
    assert p(None, 0, 64, 64, None, None, None) == 0
    assert u(FAKE, FAKE, 2, 64, 96, FAKE, None) == -2
    assert u(FAKE, None, 2, 64, 64, FAKE, None) == -1


def test_save8_and_bwd8_refusals():
    lib = _lib.load()
    s = lib.moe_grouped_gemm_swiglu_save8
    assert s(FAKE, FAKE, FAKE, FAKE, 4, 96, 64, 16, FAKE, FAKE, FAKE, None) == -2
    assert s(FAKE, FAKE, FAKE, None, 4, 64, 64, 16, FAKE, FAKE, FAKE, None) == -1
    assert s(FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, None, FAKE, None) == -1   # ab8 required
    assert s(FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, None, None) == -1   # ab8_scale required
    assert s(FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, MIS, None) == -3
    assert s(FAKE, FAKE, FAKE, FAKE, 513, 64, 64, 16, FAKE, FAKE, FAKE, None) == -1
    assert s(FAKE, FAKE, FAKE, FAKE, 4, 16384, 65536, 16, FAKE, FAKE, FAKE, None) == -1
    assert s(None, None, None, FAKE, 4, 64, 64, 0, None, None, None, None) == 0     # no rows
    g = lib.moe_grouped_gemm_swiglu_gather_save8
    assert g(FAKE, 64, FAKE, 17, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, FAKE, None) == -1
    assert g(FAKE, 8, FAKE, 1, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, FAKE, None) == -1   # cap > T*K
    assert g(FAKE, 1966081, FAKE, 8, FAKE, FAKE, FAKE, 4, 1024, 64, 16, FAKE, FAKE, FAKE, None) == -1
    assert g(FAKE, 64, None, 2, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, FAKE, None) == -1
    b = lib.moe_grouped_gemm_swiglu_bwd8
    assert b(FAKE, FAKE, FAKE, 4, 64, 96, 16, FAKE, FAKE, FAKE, FAKE, None) == -2
    assert b(FAKE, FAKE, FAKE, 4, 64, 64, 16, None, FAKE, FAKE, FAKE, None) == -1
    assert b(FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, None, FAKE, None) == -1
    assert b(FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, FAKE, MIS, None) == -3
    assert b(None, None, FAKE, 0, 64, 64, 16, None, None, None, None, None) == 0


def test_gemm4_refusals():
    lib = _lib.load()
    g = lib.moe_grouped_gemm4_swiglu
    ok = (FAKE, 64, FAKE, 2, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, None)

    def call(**kw):
        names = ("x", "T", "src", "K", "gq", "gs", "uq", "us", "off", "el", "H", "F", "cap", "h", "stream")
        a = dict(zip(names, ok), **kw)
        return g(*(a[n] for n in names))

    assert call(H=96) == -2 and call(F=96) == -2
    assert call(K=17) == -1 and call(K=0) == -1
    assert call(T=4, K=2) == -1                       # cap > T*K
    assert call(T=1966081, K=8, H=1024) == -1         # x past 0xF0000000 bytes
    assert call(el=513) == -1 and call(el=-1) == -1 and call(H=0) == -1
    assert call(H=16384, F=65536) == -1
    for n in ("x", "gq", "gs", "uq", "us", "off", "h"):
        assert call(**{n: None}) == -1, n
    for n in ("x", "src", "gq", "gs", "uq", "us", "off", "h"):
        assert call(**{n: MIS}) == -3, n
    assert call(src=None, T=0, K=0, x=None) == -1     # without src: x still required
    assert call(cap=0, x=None) == 0 and call(el=0, x=None) == 0
    d = lib.moe_grouped_gemm4
    assert d(FAKE, FAKE, FAKE, FAKE, 4, 96, 64, 16, FAKE, None) == -2
    assert d(FAKE, FAKE, None, FAKE, 4, 64, 64, 16, FAKE, None) == -1
    assert d(FAKE, FAKE, MIS, FAKE, 4, 64, 64, 16, FAKE, None) == -3
    assert d(FAKE, FAKE, FAKE, None, 4, 64, 64, 16, FAKE, None) == -1
    assert d(FAKE, FAKE, FAKE, FAKE, 4, 64, 64, -1, FAKE, None) == -1


def test_gemm4_combine_refusals():
    lib = _lib.load()
    assert lib.moe_gemm4_combine_workspace_size(10, 64) == 2560
    assert lib.moe_gemm4_combine_workspace_size(0, 64) == 0 and lib.moe_gemm4_combine_workspace_size(-1, 64) == 0
    names = ("a", "q4", "s4", "off", "el", "Kd", "N", "cap", "pos", "gates", "T", "K", "y", "out", "ws", "wsb", "st")
    ok = (FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 16, FAKE, FAKE, 8, 2, None, FAKE, FAKE, 1 << 20, None)

    def call(**kw):
        a = dict(zip(names, ok), **kw)
        return lib.moe_grouped_gemm4_combine(*(a[n] for n in names))

    assert call(Kd=96) == -2 and call(N=96) == -2
    assert call(K=0) == -1 and call(K=17) == -1 and call(T=-1) == -1 and call(T=262141) == -1
    for n in ("a", "q4", "s4", "off", "pos", "gates", "out"):
        assert call(**{n: None}) == -1, n
    for n in ("a", "q4", "s4", "off", "pos", "gates", "y", "out", "ws"):
        assert call(**{n: MIS}) == -3, n
    assert call(ws=None) == -4 and call(wsb=16 * 64 * 4 - 1) == -4
    assert call(T=0, pos=None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(_lib.MoeError):
        _lib.moe_pack8(x)
    with pytest.raises(_lib.MoeError):
        _lib.moe_unpack8(torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 2), dtype=torch.uint8))
    with pytest.raises(_lib.MoeError):
        _lib.moe_pack4(torch.zeros((1, 64, 64), dtype=torch.bfloat16))
    assert _lib.pack4_shapes(3, 192, 128) == ((3, 8, 2, 64, 16), (3, 8, 2, 64))
