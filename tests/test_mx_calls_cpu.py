"""Calls of the block-scaled operators at the edges of what moe.h allows; everything here is decided on the host."""
from routing_permute_groupgemm_amd import _lib

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
