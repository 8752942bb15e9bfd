"""Calls of the block-scaled operators at the edges of what moe.h allows; everything here is decided on the host."""
import mx_ref
import numpy as np

from routing_permute_groupgemm_amd import _lib, synth

FAKE = 0x10000  # never dereferenced


def combine(**kw):
    a = dict(a=FAKE, q4=FAKE, s4=FAKE, off=FAKE, el=4, Kd=64, N=64, cap=16, pos=FAKE, gates=FAKE, T=8, K=2, y=None,
             out=FAKE, ws=FAKE, wsb=1 << 20, st=None)
    a.update(kw)
    return _lib.load().moe_grouped_gemm4_combine(*a.values())


def test_combine_without_tokens_still_has_rows_to_write():
    """T = 0 with y: the product runs, so its operands and workspace are needed (and pos, gates and out are not)."""
    none = dict(T=0, pos=None, gates=None, out=None)
    assert combine(**none) == 0 and combine(**none, a=None, ws=None) == 0  # nothing asked for
    for n in ("a", "q4", "s4"):
        assert combine(**none, y=FAKE, **{n: None}) == -1, n
    assert combine(**none, y=FAKE, ws=None) == -4
    assert combine(**none, y=FAKE, cap=0) == 0 and combine(**none, y=FAKE, el=0) == 0 and combine(**none, y=FAKE, N=0) == 0


def test_gemm4_refuses_what_no_launch_can_hold():
    """2^32 threads and more: 2^17 row tiles of 32 rows (and one per expert) x 64 slabs of 256 columns, eight waves
    each; and 576 row tiles of 16 rows x 2^17 slabs of 128 columns, four waves each."""
    lib = _lib.load()
    up = lib.moe_grouped_gemm4_swiglu
    assert up(FAKE, 1 << 22, FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 1 << 14, 1 << 22, FAKE, None) == -1
    down = lib.moe_grouped_gemm4
    assert down(FAKE, FAKE, FAKE, FAKE, 4, 64, 1 << 14, 1 << 22, FAKE, None) == -1
    assert down(FAKE, FAKE, FAKE, FAKE, 512, 64, (1 << 24) - 64, 1024, FAKE, None) == -1
    assert combine(T=1 << 18, cap=1 << 22, N=1 << 14, wsb=1 << 40) == -1


def test_8bit_error_at_the_scale_floor():
    """Below 2^-120 the scale stays 7: a value is off by at most half a step of 2^-126, which may be all of it, and
    from 2^-120 on by at most 1/128 of the block's largest magnitude."""
    exact = np.zeros((1, 64), np.uint16)
    exact[0, :3] = 0x0040, 0x0080, 0x0001                 # 2^-127 alone rounds to even, to 0; 2^-126 is one step
    q, s = mx_ref.pack8(exact)
    assert s[0, 0] == 7 and q[0, :3].tolist() == [0, 1, 0]
    assert abs(mx_ref.unpack8(q, s)[0, 0] - 2.0 ** -127) == 2.0 ** -127 > 2.0 ** -126 / 128
    for std in (2.0 ** -118, 2.0 ** -121, 2.0 ** -125, 2.0 ** -130):
        bits = synth.f32_to_bf16_bits((np.random.default_rng(1).standard_normal((64, 256)) * std).astype(np.float32))
        q, s = mx_ref.pack8(bits)
        x, v = mx_ref.f64(bits), mx_ref.unpack8(q, s)
        m = np.repeat(np.abs(x).reshape(64, -1, 32).max(2), 32, axis=1)
        bound = np.where(m >= 2.0 ** -120, m / 128, 2.0 ** -127)
        assert (np.abs(v - x) <= bound).all()
    assert (np.abs(v - x) > m / 128).any()                # the floor is reached
