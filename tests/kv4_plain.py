"""The cache-writing and 4-bit cache operators, plainly: numpy, 64 bits, one step of each definition a line.

Shares nothing with the CUDA sources.  Where a definition rounds to fp32 (the rotation's products and sum, the
factor's product), the value is computed in 64 bits first: a product of two fp32 values is exact there, and a sum is
exact or rounded 2^-29 of a step before the rounding to fp32 that follows.
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f32(x):
    return np.asarray(x).astype(np.float32).astype(np.float64)


def bf16(x):
    """Nearest-even bf16 of float64 values that fp32 holds exactly, as float64."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def rotate(x, cos, sin, dim, interleaved, rounded=True):
    """x [..., D] float64; cos, sin [..., dim/2] float64 (fp32 values), broadcast against x's leading axes."""
    near = f32 if rounded else np.asarray
    y = np.array(x, dtype=np.float64)
    i = np.arange(dim // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
    y[..., a] = near(near(x[..., a] * cos) - near(x[..., b] * sin))
    y[..., b] = near(near(x[..., b] * cos) + near(x[..., a] * sin))
    return y


# ---- e4m3 and e2m1 ----------------------------------------------------------------------------------------
def e4m3_value(byte):
    byte = np.asarray(byte).astype(np.int64)
    e, m = byte >> 3, byte & 7
    return np.where(e == 0, m / 512.0, (1 + m / 8.0) * np.exp2(e - 7.0))


E4M3 = e4m3_value(np.arange(0x7F))  # 0 .. 448, ascending; the index is the byte


def nearest(x, values):
    """Index of the nearest of ascending `values` (ties to the even index), at most the last."""
    hi = np.clip(np.searchsorted(values, x, side="left"), 1, len(values) - 1)
    lo = hi - 1
    dl, dh = x - values[lo], values[hi] - x
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def hold(x, scale):
    """x [..., D] float64 (fp32 values) -> codes [..., D] 0..15, scale bytes [..., D/16]."""
    inv = np.float64(np.float32(1.0) / np.float32(scale))
    y = f32(x * inv).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    top = np.abs(y).max(-1)
    s = nearest(f32(top / 6.0), E4M3)
    sv = E4M3[s][..., None]
    q = np.abs(y) / np.where(sv == 0, 1.0, sv)
    code = np.where(sv == 0, 0, nearest(q, LEVELS) + 8 * np.signbit(y))
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def value(codes, scales):
    """Held values (without the call's factor) [..., D] of codes [..., D] and scale bytes [..., D/16]."""
    v = np.where(codes & 8, -1.0, 1.0) * LEVELS[codes & 7]
    return v * np.repeat(e4m3_value(scales), 16, axis=-1)


# ---- pages ---------------------------------------------------------------------------------------------------
def offsets(T, D):
    a, b = T * D // 2, T * D // 16
    return 0, a, a + b, 2 * a + b, 2 * (a + b)


def page_rows(page, T, D, values):
    """(codes [T, D], scale bytes [T, D/16]) of a page's keys or values."""
    o = offsets(T, D)
    i = 2 if values else 0
    packed = page[o[i]:o[i + 1]].reshape(T, D // 2)
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(T, D)
    return codes, page[o[i + 1]:o[i + 2]].reshape(T, D // 16)


def put_row(page, T, D, r, values, codes, scales):
    o = offsets(T, D)
    i = 2 if values else 0
    page[o[i] + r * (D // 2):o[i] + (r + 1) * (D // 2)] = codes[0::2] | (codes[1::2] << 4)
    page[o[i + 1] + r * (D // 16):o[i + 1] + (r + 1) * (D // 16)] = scales


# ---- attention ---------------------------------------------------------------------------------------------------
def unit_attention(q, k, v, sm_scale):
    """q [G, D], k and v [n, D] float64 -> out [G, D], lse [G], the largest sum |q_d k_d| * sm_scale."""
    if k.shape[0] == 0:
        return np.zeros_like(q), np.full(q.shape[0], -np.inf), 0.0
    z = (q @ k.T) * sm_scale
    m = z.max(1, keepdims=True)
    e = np.exp(z - m)
    l = e.sum(1, keepdims=True)
    return (e / l) @ v, (m + np.log(l))[:, 0], float(((np.abs(q) @ np.abs(k).T) * sm_scale).max())


def out_tolerance(D, zsum, vmax):
    """How far a fp32 attention output may be off.

    A score is a sum of D products in fp32 in some order (at most D/8 partial sums of the tensor core's rounding, two
    steps each), times a factor: at most (D/4 + 8) * 2^-24 of sum |q_d k_d| * sm_scale in the exponent.  A probability
    then has a relative error of that plus 2^-22 (exp2) plus 2^-21 (fp16 hi + lo); numerator and denominator
    each carry it, and the sums and merges add 2^-18 (their terms are rounded in partial sums of at most 64
    each)."""
    return (2 * (D / 4 + 8) * 2.0 ** -24 * zsum + 2.0 ** -18) * vmax + 1e-30


def lse_tolerance(D, zsum, lse):
    return (D / 4 + 8) * 2.0 ** -24 * zsum + 2.0 ** -18 + 2.0 ** -22 * abs(lse)
