"""Inputs, 64-bit definitions and derived tolerances of the 16-bit operators' tests."""

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half of the smallest subnormal: what a rounding near zero may be off by
FLOOR = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
# An accumulation of n products in float32 rounds (or cuts off) n times, by at most a
# whole step of 2^-23 of a partial sum, and no partial sum exceeds the sum of magnitudes.
STEP = 2.0 ** -23


def offsets_of(counts, start=0):
    c = torch.tensor([0, *counts])
    return (c.cumsum(0) + start).to(torch.int32)


def rows_of(offsets):
    o = offsets.tolist()
    return [slice(o[i], o[i + 1]) for i in range(len(o) - 1)]


def randn(*shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def check(got, ref, mag, n, what=""):
    """got against ref (64 bits), a sum of n products whose magnitudes sum to mag: n
    steps of accumulation, then one rounding to got's type."""
    err = (got.double().cpu() - ref).abs()
    acc = n * STEP * mag
    tol = acc + HALF_STEP[got.dtype] * (ref.abs() + acc) + FLOOR[got.dtype]
    bad = ~(err <= tol)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
        f"{got.double().cpu()[tuple(bad.nonzero()[0])]} for {ref[tuple(bad.nonzero()[0])]} "
        f"(allowed {tol[tuple(bad.nonzero()[0])]})")


def product64(a, w, offsets):
    """(out, sums of magnitudes) of rows inside the offsets; zeros elsewhere."""
    a, w = a.double(), w.double()
    out = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e, rows in enumerate(rows_of(offsets)):
        out[rows] = a[rows] @ w[e].T
        mag[rows] = a[rows].abs() @ w[e].abs().T
    return out, mag


def weights_grad64(dy, a, offsets, E):
    dy, a = dy.double(), a.double()
    out = torch.zeros(E, dy.shape[1], a.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e, rows in enumerate(rows_of(offsets)):
        out[e] = dy[rows].T @ a[rows]
        mag[e] = dy[rows].abs().T @ a[rows].abs()
    return out, mag


# What is lost of A x where it enters the second product as the sum of two 16-bit values:
# two roundings by half a step, relative to the row's largest (whose power of two is at
# most its magnitude), and half the smallest subnormal.
SPLIT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22 + 2.0 ** -25}


def lora64(x, a, b, ids, experts, scaling, base, dtype):
    """(out, what it may be off by before its last rounding) of moe_lora_product for
    rows with adapter ids and experts (host lists), a [L, E, r, K], b [L, E, N, r]."""
    R, N, K, r = x.shape[0], b.shape[2], x.shape[1], a.shape[2]
    out = torch.zeros(R, N, dtype=torch.float64) if base is None else base.double()
    off = torch.zeros(R, N, dtype=torch.float64)
    for l, e in {(l, e) for l, e in zip(ids, experts) if l >= 0 and e >= 0}:
        rows = [t for t in range(R) if ids[t] == l and experts[t] == e]
        s = 1.0 if scaling is None else float(scaling[l])
        al, bl, xs = a[l, e].double(), b[l, e].double(), x[rows].double()
        h = xs @ al.T * s
        h_off = (K + 1) * STEP * (xs.abs() @ al.abs().T) * abs(s) + SPLIT[dtype] * h.abs().amax(1, keepdim=True)
        out[rows] += h @ bl.T
        off[rows] += h_off @ bl.abs().T + (2 * r + 1) * STEP * ((h.abs() + h_off) @ bl.abs().T)
    return out, off + 2.0 ** -24 * out.abs()


def check_lora(got, ref, off, what=""):
    err = (got.double().cpu() - ref).abs()
    tol = off + HALF_STEP[got.dtype] * (ref.abs() + off) + FLOOR[got.dtype]
    bad = ~(err <= tol)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
        f"{got.double().cpu()[tuple(bad.nonzero()[0])]} for {ref[tuple(bad.nonzero()[0])]} "
        f"(allowed {tol[tuple(bad.nonzero()[0])]})")
