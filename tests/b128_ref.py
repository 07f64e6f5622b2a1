"""The block-scaled FP8 operators in float64 on the CPU, from their
definitions (include/llmint8.h), for the tests: E4M3 codes with one E8M0 byte
per block of 128.

E4M3 values are looked up from the format's definition; rounding to nearest
with ties to even picks between the two neighbours in the sorted table.
"""
import numpy as np
import torch

NAN_BYTE = 255
# every finite E4M3 magnitude in order: codes 0 .. 0x7e
_E4M3 = np.array([(m * 2.0 ** -9) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                  for e in range(16) for m in range(8)][:127])
EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half the subnormal step


def pitch(K):
    return (-(-K // 128) + 3) // 4 * 4


def encode(v):
    """float64 magnitudes <= 448 -> E4M3 codes 0 .. 0x7e, nearest, ties to even."""
    hi = np.searchsorted(_E4M3, v, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - _E4M3[lo], _E4M3[hi] - v
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def decode(codes):
    """uint8 E4M3 codes -> float64 (0x7f and 0xff: NaN)."""
    c = np.asarray(codes)
    mag = np.append(_E4M3, np.nan)[c & 127]
    return np.where(c & 128, -mag, mag)


def exponent(a):
    """Largest e with a * 2^e <= 448, at most 126; 0 for a = 0."""
    a = np.asarray(a, np.float64)
    m, ex = np.frexp(np.where(a > 0, a, 1.0))
    e = np.where(m <= 0.875, 9 - ex, 8 - ex)
    return np.where(a > 0, np.minimum(e, 126), 0)


def _blocks(v, rows):
    """[N,K] -> (blocks [nb, kb, rows, 128] zero-padded)."""
    N, K = v.shape
    nb, kb = -(-N // rows), -(-K // 128)
    p = np.zeros((nb * rows, kb * 128))
    p[:N, :K] = v
    return p.reshape(nb, rows, kb, 128).transpose(0, 2, 1, 3)


def quantize(v, rows):
    """float64 [N,K] -> (codes uint8 [N,K], scales uint8 [ceil(N/rows), pitch])
    in blocks of rows x 128."""
    N, K = v.shape
    p = _blocks(v, rows)
    bad = ~np.isfinite(p).all((2, 3))
    q = np.where(np.isfinite(p), p, 0.0)
    e = exponent(np.abs(q).max((2, 3)))
    c = encode(np.abs(q) * 2.0 ** e[..., None, None]) | (np.signbit(q) * 128)
    c = np.where(bad[..., None, None], 127, c)
    s = np.where(bad, NAN_BYTE, 127 - e)
    codes = c.transpose(0, 2, 1, 3).reshape(p.shape[0] * rows, -1)[:N, :K].astype(np.uint8)
    sb = np.full((s.shape[0], pitch(K)), 127, np.uint8)
    sb[:, :s.shape[1]] = s
    return codes, sb


def values(codes, scales, rows):
    """float64 values of codes [N,K] under scales [ceil(N/rows), pitch]."""
    N, K = codes.shape
    s = np.where(scales == NAN_BYTE, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    s = s.repeat(rows, 0)[:N].repeat(128, 1)[:, :K]
    return decode(codes) * s


def to64(t):
    return t.detach().to("cpu").double().numpy()


def f8_sum_bound(K, S):
    """How far a length-K sum by the fp8 matrix instructions may be from the
    exact one, S = sum of its products' magnitudes.  Groups of eight products
    are summed with 13 bits below the largest (the rest dropped), and the
    groups and the accumulator with about 24: per instruction
    7 * 2^-13 * (its products) + 11 * 2^-24 * (those + |accumulator|), over
    ceil(K/32) instructions at most."""
    return (7 * 2.0 ** -13 + 11 * 2.0 ** -24 * -(-K // 32)) * S


def product_bound(K, S, ref, dtype, wave_sums=0):
    """The bound of an output: the sum's, fp32 additions of partial sums and
    the bias, and one rounding to the output type."""
    e = f8_sum_bound(K, S) + (wave_sums + 2) * 2.0 ** -24 * (S + np.abs(ref))
    return e + EPS[dtype] * (np.abs(ref) + e) + TINY[dtype]
