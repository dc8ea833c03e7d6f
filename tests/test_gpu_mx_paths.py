"""Branches of the microscaled operators that only some sizes reach: forwards
above 2048 slots, K splits (of single CTAs, of pairs, and of a forward's down
product), the wide slot sum, norms between 4096 and 8192, the bulk quantiser in
every type, long rows, bad offsets in every shape of the product.

Tolerances as derived in test_gpu_mx.py, but for the wide slot sum: with I = 128
one activation whose code falls the other way at a tie moves a whole token by
more than that forward bound (3e-2 rms for one at 2e-7 of a tie), so its bound
follows each activation (forward_with_bound).  A product may have sixteen K splits, so
sixteen sums stand where that bound has eight: |err| <= (K / 32 + 18) 2^-22 S +
half an ulp of the output.
"""

import numpy as np
import pytest
import torch

from moe_helpers import check_forward
from oracle import mx_oracle as mx
from test_gpu_mx import (HALF_ULP, check_norm, cuda_mx, done, forward_case, forward_ref, np64,
                         product_case, rnd)

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("weight_quantized_moe_gb300")


def launches(call):
    """(result, kernel launches) of a call."""
    lib = mq.binding.lib()
    before = lib.mq_kernel_launch_count()
    result = call()
    return result, lib.mq_kernel_launch_count() - before


def is_split(S, E, K, N, bits):
    """Whether a product of these sizes splits K: a second launch joins the sums."""
    a = torch.zeros(S, K * bits // 8, dtype=torch.uint8, device="cuda")
    w = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    scales = [torch.zeros(*t.shape[:-1], K // 32, dtype=torch.uint8, device="cuda") for t in (a, w)]
    _, n = launches(lambda: mq.moe_mx_product(a, scales[0], w, scales[1], expert_offsets=offs, a_bits=bits))
    done()
    return n == 2


def check_long_product(got, ref, mag, K):
    tol = (K / 32 + 18) * 2.0 ** -22 * mag + HALF_ULP[got.dtype] * np.abs(ref)
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), (err / tol).max()


def forward_with_bound(c, bits):
    """(reference, largest error) of a forward, element by element.

    h is a product: |dh| <= (H / 32 + 10) 2^-22 sum |a| |w|.  silu is g / (1 + exp(-g))
    with |silu'| <= 1.1, the exponential within 2 + 1.2 |g| units of 2^-23, the
    quotient within two and three roundings: 2^-18 of the result where |g| <= 20.  So
    an activation is known to d = 1.1 dg |u| + |silu| du + 2^-18 |act|, and its code
    may be any that act - d .. act + d take under the scales of the block's maximum
    minus and plus d.  What that leaves open, times |w2|, is added to the second
    product's own bound (at most sixteen K splits) and the sum over k slots."""
    qa, sa, q13, s13, q2, s2, tw, ids = [t.cpu().numpy() for t in c]
    a = mx.mx_dequantize(qa, sa, bits)
    w13, w2 = mx.mx_dequantize(q13, s13, 4), mx.mx_dequantize(q2, s2, 4)
    E, H, I = w2.shape
    ref, tol = np.zeros((len(a), H)), np.zeros((len(a), H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        h = a[t] @ w13[e].T
        dh = (H / 32 + 10) * 2.0 ** -22 * (np.abs(a[t]) @ np.abs(w13[e]).T)
        g, u, dg, du = h[:, :I], h[:, I:], dh[:, :I], dh[:, I:]
        assert np.abs(g).max() <= 20
        silu = g / (1 + np.exp(-g))
        act = silu * u
        d = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 2.0 ** -18 * np.abs(act)
        blocks = lambda v: v.reshape(len(t), -1, 32)  # noqa: E731
        ends = []
        for sc in (mx.scale_codes(np.maximum(blocks(np.abs(act) - d).max(-1), 0), bits),
                   mx.scale_codes(blocks(np.abs(act) + d).max(-1), bits)):
            for v in (act - d, act + d):
                ends.append(mx.mx_dequantize(mx.pack(mx.elements(v, sc, bits), bits), sc, bits))
        lo, hi = np.minimum.reduce(ends), np.maximum.reduce(ends)
        b = mx.mx_dequantize(*mx.mx_quantize(act, bits), bits)
        w = np.abs(tw[t, j])[:, None].astype(np.float64)
        np.add.at(ref, t, (b @ w2[e].T) * tw[t, j][:, None].astype(np.float64))
        most = np.maximum(np.abs(lo), np.abs(hi))
        np.add.at(tol, t, w * (np.maximum(hi - b, b - lo) @ np.abs(w2[e]).T
                               + (I / 32 + 18 + 2 * ids.shape[1]) * 2.0 ** -22 * (most @ np.abs(w2[e]).T)))
    return ref, tol


def check_bounded(got, ref, tol):
    tol = tol + HALF_ULP[got.dtype] * (np.abs(ref) + tol)
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25      # subnormal outputs
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), (err / np.maximum(tol, 1e-300)).max()


# ------------------------------------------------------------------- forward --
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,k", [(1024, 2), (683, 3), (1025, 2), (2049, 1), (1500, 2)])
def test_forward_around_2048_slots(T, k, bits):
    """Slots are put in order in one launch up to 2048, by the align kernel and
    a gather above: uneven loads, an expert without a token, ids out of range."""
    E, H, I = 6, 256, 384
    c = forward_case(T, E, k, H, I, bits, seed=T)
    ids = c[7]
    ids[ids == 4] = 1                       # expert 4 gets nothing, 1 twice as much
    ids[5, 0], ids[T - 1, k - 1], ids[T // 2] = -1, E, 1000
    got, n = launches(lambda: mq.moe_mx_forward(*c, a_bits=bits))
    assert mq.mq_device_status() == mq.MQ_DEV_BAD_EXPERT_ID
    assert n == (5 if T * k > 2048 else 4)
    check_forward(np64(got), forward_ref(*c, bits), what=f"mx forward {T} {k} {bits}")
    assert not got[T // 2].any()            # (all of its slots are left out)


@pytest.mark.parametrize("E,loads", [(3, "one"), (40, "even"), (40, "zipf")])
def test_forward_above_2048_slots_loads(E, loads):
    """All tokens on one expert, a few rows each, some experts empty."""
    T, k, H, I = 2500, 1, 128, 256
    c = forward_case(T, E, k, H, I, 8, seed=E)
    g = torch.Generator().manual_seed(1)
    if loads == "one":
        c[7].fill_(E - 1)
    elif loads == "zipf":
        p = 1.0 / torch.arange(1, E + 1) ** 2
        c[7].copy_(torch.multinomial(p, T * k, replacement=True, generator=g).view(T, k))
    got = mq.moe_mx_forward(*c, a_bits=8)
    done()
    check_forward(np64(got), forward_ref(*c, 8), what=f"mx forward E={E} {loads}")


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 2, 2, 256, 8192), (3, 4, 2, 384, 14336), (17, 6, 1, 256, 4096),
                                       (20, 4, 2, 128, 6144), (500, 4, 2, 128, 4096)])
def test_forward_with_k_splits(T, E, k, H, I, bits):
    """The down product's partial sums of several splits, joined in the slot sum."""
    assert is_split(T * k, E, I, H, bits)
    c = forward_case(T, E, k, H, I, bits, seed=T + I)
    if T > 1:
        c[7][T // 2, 0] = -1
    got = mq.moe_mx_forward(*c, a_bits=bits)
    assert mq.mq_device_status() == (mq.MQ_DEV_BAD_EXPERT_ID if T > 1 else 0)
    check_forward(np64(got), forward_ref(*c, bits), what=f"mx forward {T} {E} {k} {H} {I} {bits}")


@pytest.mark.parametrize("T,k,H,out_dtype", [(620, 1, 4096, torch.bfloat16), (640, 3, 4224, torch.float16),
                                             (1300, 2, 4224, torch.bfloat16)])
def test_forward_wide_slot_sum(T, k, H, out_dtype):
    c = forward_case(T, 3, k, H, 128, 8, seed=H)
    c[7][7, 0] = 3
    got = mq.moe_mx_forward(*c, a_bits=8, out_dtype=out_dtype)
    assert mq.mq_device_status() == mq.MQ_DEV_BAD_EXPERT_ID
    check_bounded(got, *forward_with_bound(c, 8))


# ------------------------------------------------------------------- product --
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,E,K,N,loads", [(256, 1, 4096, 256, [256]), (256, 1, 4096, 257, [256]),
                                           (200, 2, 4096, 300, [199, 1]), (120, 1, 14336, 128, [120])])
def test_product_pairs_with_k_splits(R, E, K, N, loads, bits):
    qa, sa, qw, sw, offs, (ref, mag) = product_case(R, E, K, N, bits, loads, seed=R)
    got, n = launches(lambda: mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs, a_bits=bits))
    done()
    assert n == 2
    check_long_product(got, ref, mag, K)


def random_weights(E, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
            torch.randint(116, 126, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,E,K,N,split", [
    (1100, 1, 14336, 256, False),    # pairs, 28 scale slots of a ring of 4 per unit
    (1100, 16, 14336, 128, False),   # single CTAs, 96-row tiles, the same
    (1100, 40, 14336, 100, False),
    (1100, 3, 14208, 128, False),    # rows that end inside a stage and a scale slot
    (3, 1, 65536, 40, True),         # eight slots per split
    (20, 1, 65536, 40, True),
    (90, 1, 65408, 40, True),
])
def test_product_long_rows(R, E, K, N, split, bits):
    g = torch.Generator().manual_seed(R + K)
    loads = np.bincount(torch.randint(0, E, (R,), generator=g).numpy(), minlength=E)
    offs = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)
    qa, sa = mq.moe_quantize_mx(rnd(R, K, seed=R).cuda(), bits=bits)
    qw, sw = random_weights(E, N, K, seed=N)
    got, n = launches(lambda: mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=torch.from_numpy(offs).cuda(),
                                                a_bits=bits, out_dtype=torch.float32))
    done()
    assert n == (2 if split else 1)
    cpu = lambda t: t.cpu().numpy()  # noqa: E731
    av = mx.mx_dequantize(cpu(qa), cpu(sa), bits)
    for e in range(E):
        s = slice(offs[e], offs[e + 1])
        wv = mx.mx_dequantize(cpu(qw[e]), cpu(sw[e]), 4)
        check_long_product(got[s], av[s] @ wv.T, np.abs(av[s]) @ np.abs(wv).T, K)


BAD_OFFSETS = [
    lambda R: [0, R // 2, R // 4, R], lambda R: [-4, 3, R // 2, R], lambda R: [0, 5, 9, 1 << 30],
    lambda R: [R + 1, R + 2, R + 3, R + 3], lambda R: [0, -(1 << 31), (1 << 31) - 1, R],
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,K,N", [(20, 128, 64), (20, 4096, 64), (20, 4096, 65), (400, 256, 96), (400, 4096, 97)])
@pytest.mark.parametrize("bad", range(len(BAD_OFFSETS)))
def test_bad_offsets_stay_inside_the_arrays(R, K, N, bits, bad):
    """Single CTAs, pairs, both with and without K splits: the status is set, and
    nothing outside the output is written."""
    qa, sa = mq.moe_quantize_mx(rnd(R, K, seed=1).cuda(), bits=bits)
    qw, sw = random_weights(3, N, K, seed=2)
    around = torch.full((R + 16, N), 7.0, dtype=torch.float32, device="cuda")
    offs = torch.tensor(BAD_OFFSETS[bad](R), dtype=torch.int64).to(torch.int32).cuda()
    mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs, a_bits=bits, out=around[8:R + 8])
    assert mq.mq_device_status() == mq.MQ_DEV_BAD_OFFSETS
    assert (around[:8] == 7).all() and (around[R + 8:] == 7).all()


# ------------------------------------------------------- norm and quantiser --
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,H", [(3, 4128), (2, 5120), (5, 7168), (3, 8160), (2, 8192)])
def test_norm_between_4096_and_8192(dtype, bits, T, H):
    x = rnd(T, H, seed=T).to(dtype).cuda()
    res = (rnd(T, H, seed=T + 1) * torch.exp(rnd(H, seed=5))).to(dtype).cuda()
    w = (1 + 0.2 * rnd(H, seed=6)).cuda()
    got = mq.moe_rmsnorm_mx(x, w, eps=1e-5, residual=res, bits=bits, want_y=True)
    done()
    check_norm(x, res, w, 1e-5, bits, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("strided", [False, True])
def test_quantise_bulk_bit_exact(dtype, bits, strided):
    """Inputs large enough for several vectors per thread; the last CTA is not full."""
    rows, cols = 1301, 2080
    wide = cols + 96 if strided else cols
    x = (rnd(rows, wide, seed=bits) * torch.exp(2 * rnd(wide, seed=9))).to(dtype)
    x[17, 64:96] = 0
    x[rows - 1, wide - 1] = float("inf")
    x = x.cuda()[:, wide - cols:]
    q, s = mq.moe_quantize_mx(x, bits=bits)
    done()
    oq, os_ = mx.mx_quantize(np64(x), bits)
    assert np.array_equal(s.cpu().numpy(), os_)
    assert np.array_equal(q.cpu().numpy(), oq)


def test_quantised_values_pass_through_the_inverse_in_bulk():
    x = rnd(3000, 1408, seed=2).cuda()
    for bits in (4, 8):
        q, s = mq.moe_quantize_mx(x, bits=bits)
        want = mx.mx_dequantize(q.cpu().numpy(), s.cpu().numpy(), bits)
        for dtype in (torch.float32, torch.bfloat16, torch.float16):
            got = mq.moe_dequantize_mx(q, s, bits=bits, dtype=dtype)
            done()
            assert torch.equal(got.cpu(), torch.from_numpy(want).float().to(dtype))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,E", [(16, 1), (17, 1), (32, 1), (33, 1), (44, 1), (45, 1), (46, 2), (47, 2),
                                 (150, 8), (151, 8), (222, 8), (223, 8), (471, 40), (633, 40)])
def test_product_at_the_borders_of_the_tile_choice(R, E, bits):
    """Where the rows per tile change, with even loads and with most rows on one expert."""
    K, N = 384, 260
    even = [R // E + (e < R % E) for e in range(E)]
    one = [0] * (E - 1) + [R] if E > 1 else even
    for loads in (even, one):
        qa, sa, qw, sw, offs, (ref, mag) = product_case(R, E, K, N, bits, loads, seed=R)
        got = mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs, a_bits=bits, out_dtype=torch.float32)
        done()
        check_long_product(got, ref, mag, K)
