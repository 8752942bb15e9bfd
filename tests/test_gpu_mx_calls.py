"""Calls of the block-scaled operators that moe.h allows at the edges of their arguments."""
import pytest
import torch

from routing_permute_groupgemm_amd import _lib

pytestmark = pytest.mark.gpu


def normal(seed, *shape, std=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


@pytest.mark.parametrize("rows", [1, 70])
def test_combine_without_tokens_writes_the_rows(rows):
    """No token (an empty batch beside rows of other GPUs): y is moe_grouped_gemm4's, which rounds the same sums."""
    a, w = normal(1, rows, 192), _lib.moe_pack4(normal(2, 2, 192, 128, std=0.05))
    offsets = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    y = torch.full((rows + 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    out = _lib.moe_grouped_gemm4_combine(a, w, offsets, rows, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                                         torch.empty((0, 2), device="cuda"), y=y)
    assert out.shape == (0, 128)
    assert torch.equal(y[:rows], _lib.moe_grouped_gemm4(a, w, offsets, rows)) and (y[rows:] == 5.0).all()


def test_pack8_of_a_buffer_past_2_36_values():
    """2^24 rows of 4096 with three of them routed: a grid of as many workgroups as the buffer has chunks would
    have 2^32 threads, which no launch may have."""
    x = normal(3, 3, 4096)
    offsets = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    want_q, want_s = _lib.moe_pack8(x)
    q, s = torch.full((4, 4096), 55, dtype=torch.int8, device="cuda"), torch.full((4, 128), 9, dtype=torch.uint8,
                                                                                  device="cuda")
    v = torch.full((4, 4096), 5.0, dtype=torch.bfloat16, device="cuda")
    lib, st = _lib.load(), torch.cuda.current_stream().cuda_stream
    # only the routed rows are touched, so the buffers need hold no more
    assert lib.moe_pack8(x.data_ptr(), 1 << 24, 4096, offsets.data_ptr(), 1, q.data_ptr(), s.data_ptr(), st) == 0
    assert lib.moe_unpack8(q.data_ptr(), s.data_ptr(), 1 << 24, 4096, offsets.data_ptr(), 1, v.data_ptr(), st) == 0
    assert torch.equal(q[:3], want_q) and torch.equal(s[:3], want_s)
    assert torch.equal(v[:3], _lib.moe_unpack8(want_q, want_s))
    assert (q[3] == 55).all() and (s[3] == 9).all() and (v[3] == 5.0).all()


def test_pack8_of_2_36_values():
    """The same sizes with every row there: the rows behind the first 2^36 - 4096 values are a workgroup's second
    step, and are packed and unpacked like the others."""
    torch.cuda.empty_cache()
    rows, cols = (1 << 24) + 3, 4096
    need = rows * cols * 3 + rows * cols // 32
    if torch.cuda.mem_get_info()[0] < need + (12 << 30):
        pytest.skip(f"needs {need >> 30} GiB of free memory")
    x = torch.full((rows, cols), 1.0, dtype=torch.bfloat16, device="cuda")
    probe = [0, 1, 1 << 23, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, rows - 1]
    want = normal(4, len(probe), cols)
    x[probe] = want
    wq, ws = _lib.moe_pack8(want)
    print(f"[mx] pack8 of {rows} x {cols}", flush=True)
    q, s = _lib.moe_pack8(x)
    torch.cuda.synchronize()
    assert torch.equal(q[probe], wq) and torch.equal(s[probe], ws)
    x.fill_(3.0)
    print("[mx] unpack8", flush=True)
    _lib.moe_unpack8(q, s, x)
    torch.cuda.synchronize()
    assert torch.equal(x[probe], _lib.moe_unpack8(wq, ws))
    x[probe], q[probe], s[probe] = 1.0, 64, 127  # 1.0 is 64 steps of 2^-6
    for lo in range(0, rows, 1 << 20):
        part = slice(lo, lo + (1 << 20))
        for t, v in ((x, 1.0), (q, 64), (s, 127)):
            a, b = torch.aminmax(t[part])
            assert float(a) == float(b) == v, (lo, v)
    del x, q, s
    torch.cuda.empty_cache()


def test_gemm4_bits_of_a_row_go_by_the_sizes_alone():
    """Two rows an expert: their bits stay when the other experts' rows change, and under another capacity, which
    takes another kernel with another order of the sum, they differ by the roundings of two fp32 sums at most."""
    E, Kd, N = 16, 2048, 1024
    a, w = normal(5, 2 * E, Kd), _lib.moe_pack4(normal(6, E, Kd, N, std=0.05))
    offsets = torch.arange(0, 2 * E + 1, 2, dtype=torch.int32, device="cuda")
    got = _lib.moe_grouped_gemm4(a, w, offsets, 2 * E)
    other = a.clone()
    other[:6], other[8:] = 100.0, float("nan")
    assert torch.equal(_lib.moe_grouped_gemm4(other, w, offsets, 2 * E)[6:8], got[6:8])
    # an expert's two rows alone, and all rows under the capacity of many more
    alone = torch.tensor([0] * 4 + [2] * 13, dtype=torch.int32, device="cuda")
    one = _lib.moe_grouped_gemm4(a[6:8], w, alone, 2)
    cap = 40 * E
    many = _lib.moe_grouped_gemm4(torch.cat((a, a.new_zeros((cap - 2 * E, Kd)))), w, offsets, cap)
    dense = _lib.moe_unpack4(*w, Kd)
    want = torch.stack([a[r].double() @ dense[r // 2].double() for r in range(2 * E)])
    tol = torch.stack([Kd * 2.0 ** -24 * (a[r].double().abs() @ dense[r // 2].double().abs()) for r in range(2 * E)])
    for c, rows in ((got, slice(0, 2 * E)), (one, slice(6, 8)), (many[:2 * E], slice(0, 2 * E))):
        assert ((c.double() - want[rows]).abs() <= tol[rows] + 2.0 ** -8 * want[rows].abs() + 1e-37).all()


@pytest.mark.parametrize("H,E,rows,F", [(512, 8, 64, 2304), (576, 8, 64, 2304), (2048, 4, 250, 1024), (2112, 4, 120, 1024),
                                        (2112, 4, 250, 2048), (3648, 7, 60, 1984), (4096, 6, 64, 2048),
                                        (4160, 3, 64, 2048), (4160, 7, 130, 512)])
def test_save8_on_both_sides_of_its_tile_rule(H, E, rows, F):
    """More panels of weights than CUs and fewer, contractions at the rule's borders: h and the bytes are the bf16
    call's, bit for bit, whichever tiles the sizes choose."""
    x, w = normal(7, E * rows, H), [normal(8 + i, E, H, F, std=0.02) for i in range(2)]
    offsets = torch.arange(0, E * rows + 1, rows, dtype=torch.int32, device="cuda")
    offsets[1:-1] += 3  # uneven
    n = E * rows
    ab = torch.empty((n, 2 * F), dtype=torch.bfloat16, device="cuda")
    h = _lib.moe_grouped_gemm_swiglu(x, w[0], w[1], offsets, n, ab_save=ab)
    q, s = _lib.moe_pack8(ab)
    src = torch.arange(n, dtype=torch.int32, device="cuda")
    for got in (_lib.moe_grouped_gemm_swiglu_save8(x, w[0], w[1], offsets, n),
                _lib.moe_grouped_gemm_swiglu_gather_save8(x, src, 1, w[0], w[1], offsets, n)):
        for a, b in zip(got, (h, q, s)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("Kd,N", [(192, 2112), (1408, 2112)])
def test_gemm4_of_many_experts_with_a_row_or_two(Kd, N):
    """16-row tiles of waves with columns of their own, for both products (100 experts of up to three rows, more
    column tiles than the split kernel takes), with weights that stay in the last-level cache and that do not."""
    E = 100
    n = [(5 * i) % 4 if i % 7 else 0 for i in range(E)]
    off = torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32)
    R = sum(n)
    assert R <= 2 * E
    x, w = normal(11, R, Kd), [normal(12 + i, E, Kd, N, std=0.02) for i in range(2)]
    packed = [_lib.moe_pack4(m) for m in w]
    del w
    h = _lib.moe_grouped_gemm4_swiglu(x, None, None, packed[0], packed[1], off, R)
    c = _lib.moe_grouped_gemm4(x, packed[0], off, R)
    vals, ends = [_lib.moe_unpack4(*p, Kd) for p in packed], off.tolist()
    for j in range(E):
        xr = x[ends[j]:ends[j + 1]].double()
        a, b = (xr @ v[j].double() for v in vals)
        # fp32 sums of Kd products, the sigmoid (2^-18 with what follows it) and one rounding to bf16
        ea, eb = (Kd * 2.0 ** -24 * (xr.abs() @ v[j].double().abs()) for v in vals)
        assert ((c[ends[j]:ends[j + 1]].double() - a).abs() <= ea + 2.0 ** -8 * a.abs()).all(), j
        s = torch.sigmoid(a)
        want = a * s * b
        tol = 1.1 * ea * b.abs() + (a * s).abs() * eb + 1.1 * ea * eb + (2.0 ** -8 + 2.0 ** -18) * want.abs() + 1e-37
        assert ((h[ends[j]:ends[j + 1]].double() - want).abs() <= tol).all(), j
