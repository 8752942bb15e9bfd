"""Block-scaled storage written from its definition in numpy float64 (no code shared with the HIP side)."""
import numpy as np

from routing_permute_groupgemm_amd import synth

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(bits):
    return synth.bf16_bits_to_f32(bits).astype(np.float64)


def biased_exponent(bits):
    """Of bf16 bit patterns (0 for zeros and denormals, 255 for infinities and NaN)."""
    return ((bits >> 7) & 0xFF).astype(np.int64)


def pack8(bits):
    """bf16 bits [rows, cols] -> (q int8, scale uint8 [rows, cols/32])."""
    rows, cols = bits.shape
    blk = bits.reshape(rows, cols // 32, 32)
    top = biased_exponent((blk & 0x7FFF).max(axis=2))
    s = np.maximum(top, 7)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.clip(np.rint(f64(blk) * np.ldexp(1.0, 133 - s)[..., None]), -127, 127)
    q = np.where((s == 255)[..., None], 0, q)
    return q.reshape(rows, cols).astype(np.int8), s.astype(np.uint8)


def unpack8(q, s):
    """-> float64 values."""
    step = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 133))
    return (q.astype(np.float64).reshape(q.shape[0], -1, 32) * step[..., None]).reshape(q.shape)


def codes4(bits):
    """bf16 bits [E, Kd, N] -> (codes uint8 [E, Kd, N], scale int64 [E, Kd/32, N])."""
    E, Kd, N = bits.shape
    blk = bits.reshape(E, Kd // 32, 32, N)
    top = biased_exponent((blk & 0x7FFF).max(axis=2))
    s = np.where(top == 255, 255, np.maximum(top - 2, 2))
    with np.errstate(invalid="ignore", over="ignore"):
        u = np.abs(f64(blk)) * np.ldexp(1.0, 127 - s)[:, :, None]
    u = np.where((s == 255)[:, :, None], 0.0, u)
    # nearest code, a tie to the even one, saturating
    c = np.zeros(u.shape, np.int64)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        c += (u >= mid) if i % 2 else (u > mid)
    c += 8 * ((blk >> 15) & 1) * (s != 255)[:, :, None]
    return c.reshape(E, Kd, N).astype(np.uint8), s


def values4(codes, s):
    """-> float64 [E, Kd, N]."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    step = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(step, 32, axis=1)


def layout4(codes, s):
    """The stored form, one entry at a time by the header's formula."""
    E, Kd, N = codes.shape
    KT = -(-Kd // 128)
    q4 = np.zeros((E, N // 16, KT, 64, 16), np.uint8)
    s4 = np.zeros((E, N // 16, KT, 64), np.uint8)
    n = np.arange(N)
    for k in range(Kd):
        kt, g, t, i = k // 128, k % 128 // 32, k % 32 // 8, k % 8 // 2
        q4[:, n // 16, kt, 16 * g + n % 16, 4 * t + i] |= codes[:, k] << (4 * (k & 1))
        s4[:, n // 16, kt, 16 * g + n % 16] = s[:, k // 32]
    return q4, s4
