"""Plain numpy restatement, in 64 bits, of the microscaled (MX) operators.

Blocks of 32 elements, E2M1 (4 bits) or E4M3 (8 bits), with one E8M0 scale
each; the residual + RMS norm that writes such rows; the product of rows
grouped by expert with 4-bit weights; the expert MLP on such rows.  Test
infrastructure only: nothing here is shared with the CUDA path.
"""

from __future__ import annotations

import numpy as np

BLOCK = 32

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def _e4m3_table():
    t = np.zeros(127)
    for c in range(127):  # code 127 is NaN
        e, m = c >> 3, c & 7
        t[c] = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return t


E4M3 = _e4m3_table()


def element_values(bits):
    """Non-negative element values by code."""
    return E2M1 if bits == 4 else E4M3


def round_to_element(v, bits):
    """Codes (sign bit included) of v rounded to the nearest element, ties to
    the even code, clamped to the largest."""
    table = element_values(bits)
    m = np.abs(v)
    hi = np.searchsorted(table, m, side="left").clip(max=len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - table[lo], table[hi] - m
    pick_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    code = np.where(m >= table[-1], len(table) - 1, np.where(pick_lo, lo, hi))
    return (code + np.signbit(v) * (8 if bits == 4 else 128)).astype(np.uint8)


def scale_codes(amax, bits):
    """E8M0 codes for the largest magnitudes of blocks."""
    amax = np.asarray(amax, dtype=np.float64)
    emax = 2 if bits == 4 else 8
    fine = np.isfinite(amax)
    e = np.frexp(np.where(fine & (amax > 0), amax, 1.0))[1] - 1 - emax
    e = np.where(amax == 0, -127, e).clip(-127, 127)
    return np.where(fine, e + 127, 255).astype(np.uint8)


def elements(v, scale, bits):
    """Element codes of v [..., K] under given scale codes [..., K / 32]."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    s = np.exp2(scale.astype(np.float64) - 127)[..., None]
    t = np.where((scale == 255)[..., None], 0.0, np.where(np.isfinite(b), b, 0.0) / s)
    return round_to_element(t, bits).reshape(v.shape)


def pack(codes, bits):
    return codes if bits == 8 else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def mx_quantize(v, bits):
    """[..., K] -> (packed codes, scale codes)."""
    v = np.asarray(v, dtype=np.float64)
    b = np.abs(v.reshape(*v.shape[:-1], -1, BLOCK))
    amax = np.where(np.isfinite(b).all(-1), np.where(np.isfinite(b), b, 0).max(-1), np.inf)
    scale = scale_codes(amax, bits)
    return pack(elements(v, scale, bits), bits), scale


def mx_dequantize(q, scale, bits):
    """The float64 values that codes and scale codes stand for."""
    table = element_values(bits)
    full = np.concatenate([table, -table]) if bits == 4 else np.concatenate(
        [table, [np.nan], -table, [np.nan]])
    if bits == 4:
        codes = np.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=np.uint8)
        codes[..., 0::2] = q & 15
        codes[..., 1::2] = q >> 4
    else:
        codes = q
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return full[codes] * np.repeat(s, BLOCK, axis=-1)


def rmsnorm(x, residual, weight, eps):
    """(h, y) of the residual addition and the norm."""
    h = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    return h, y


def mx_product(a, w, offsets):
    """a [R, K], w [E, N, K] (values), offsets [E + 1] -> [R, N]; rows outside
    are NaN.  Also the sums of magnitudes, for error bounds."""
    out = np.full((a.shape[0], w.shape[1]), np.nan)
    mag = np.zeros_like(out)
    for e in range(w.shape[0]):
        s = slice(offsets[e], offsets[e + 1])
        out[s] = a[s] @ w[e].T
        mag[s] = np.abs(a[s]) @ np.abs(w[e]).T
    return out, mag


def mx_forward(a, w13, w2, topk_w, topk_ids, bits):
    """Expert MLP: a [T, H], w13 [E, 2I, H], w2 [E, H, I] (values)."""
    E, H, I = w2.shape
    out = np.zeros((a.shape[0], H))
    for e in range(E):
        t, j = np.nonzero(topk_ids == e)
        if len(t) == 0:
            continue
        h = a[t] @ w13[e].T
        with np.errstate(over="ignore"):
            act = h[:, :I] / (1 + np.exp(-h[:, :I])) * h[:, I:]
        act = mx_dequantize(*mx_quantize(act, bits), bits)
        np.add.at(out, t, (act @ w2[e].T) * topk_w[t, j][:, None].astype(np.float64))
    return out
