"""GPU parity of the microscaled operators against the 64-bit oracle.

Tolerances, derived:
* codes and scales of moe_quantize_mx: bit for bit (every step but the
  element rounding is exact); moe_dequantize_mx: one rounding of an exact value.
* moe_rmsnorm_mx: its float32 y differs from the exact one by at most
  DELTA = 64 * 2^-24 relative: a thread adds at most 32 squares and the joins
  are 10 more additions (42 half-ulps on the sum, half of that on its root),
  rsqrt 2 ulp, the division, the residual addition and two multiplications
  one rounding each.  A 16-bit output then lies within its own half ulp; a
  scale lies between those of the block's maximum times 1 -+ DELTA, and an
  element between those of y (1 - DELTA) and y (1 + DELTA) under that scale.
* moe_mx_product: products of codes and scales are exact; K / 32 instructions
  at most add to the float32 accumulator, each within 2^-22 of the largest
  partial sum, itself at most S = sum |a| |w|; a K split adds 8 more sums.
  |err| <= (K / 32 + 10) 2^-22 S + half an ulp of the output.
* moe_mx_forward: the library's forward bound, 1e-2 rms + |ref| 2^-8 (a
  requantised activation at a rounding tie may go either way).
"""

import numpy as np
import pytest
import torch

from moe_helpers import check_forward
from oracle import mx_oracle as mx

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("weight_quantized_moe_gb300")

DELTA = 64 * 2.0 ** -24
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def rnd(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * std


def np64(t):
    return t.detach().double().cpu().numpy()


def cuda_mx(v, bits):
    """Oracle-quantised values as device codes and scales."""
    q, s = mx.mx_quantize(v, bits)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()


def done():
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0


# ----------------------------------------------------------------- quantiser --
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (2, 5, 64), (64,), (517, 1408), (33, 4096)])
def test_quantise_bit_exact(dtype, bits, shape):
    x = (rnd(*shape, seed=len(shape) + bits) * torch.exp(2 * rnd(shape[-1], seed=9))).to(dtype).cuda()
    q, s = mq.moe_quantize_mx(x, bits=bits)
    done()
    oq, os_ = mx.mx_quantize(np64(x), bits)
    assert np.array_equal(s.cpu().numpy(), os_)
    assert np.array_equal(q.cpu().numpy(), oq)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantise_special_values(bits):
    """Ties, zeros of both signs, subnormals, the largest floats, infinities
    and NaN, each in a block of its own."""
    rows = np.zeros((9, 32), dtype=np.float32)
    rows[0, :16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6]
    rows[1, :8] = [448, 1.0625, 1.1875, 17, 19, 2 ** -10, 3 * 2 ** -10, -464]
    rows[2, 0] = -0.0
    rows[3, :4] = [1e-45, -3e-45, 1e-40, -1.1e-38]
    rows[4, :3] = [3.4028235e38, -3e38, 1.0]
    rows[5, 7] = np.inf
    rows[6, 31] = -np.inf
    rows[7, 0] = np.nan
    rows[8] = 2.0 ** -126
    q, s = mq.moe_quantize_mx(torch.from_numpy(rows).cuda(), bits=bits)
    done()
    oq, os_ = mx.mx_quantize(rows, bits)
    assert np.array_equal(s.cpu().numpy(), os_)
    assert np.array_equal(q.cpu().numpy(), oq)


def test_quantise_strided_rows_and_empty():
    wide = rnd(40, 160, seed=3).to(torch.bfloat16).cuda()
    for x in (wide[:, 32:96], wide[::3, :64], wide.view(4, 10, 160)[..., :32]):
        q, s = mq.moe_quantize_mx(x, bits=4)
        oq, os_ = mx.mx_quantize(np64(x), 4)
        assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), os_)
    q, s = mq.moe_quantize_mx(wide[:0], bits=8)
    assert q.shape == (0, 160) and s.shape == (0, 5)
    done()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_dequantise_every_code(bits, dtype):
    codes = np.arange(256, dtype=np.uint8).reshape(1, 256).repeat(256, 0)
    n = 512 if bits == 4 else 256
    scale = np.arange(256, dtype=np.uint8)[:, None].repeat(n // 32, 1)
    got = mq.moe_dequantize_mx(torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(),
                               bits=bits, dtype=dtype).cpu()
    done()
    want = torch.from_numpy(mx.mx_dequantize(codes, scale, bits)).to(torch.float32).to(dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))


# ---------------------------------------------------------------------- norm --
def check_norm(x, res, w, eps, bits, got):
    q, s, r, y = got
    h, y64 = mx.rmsnorm(np64(x), None if res is None else np64(res), np64(w), eps)
    if r is not None:
        want = torch.from_numpy(h).float().to(x.dtype)
        assert torch.equal(r.cpu(), want)      # one float32 addition, one rounding
    if y is not None:
        tol = np.abs(y64) * (HALF_ULP[x.dtype] + DELTA) + 2.0 ** -24
        assert np.all(np.abs(np64(y) - y64) <= tol)
    amax = np.abs(y64).reshape(*y64.shape[:-1], -1, 32).max(-1)
    sc = s.cpu().numpy()
    lo, hi = mx.scale_codes(amax * (1 - DELTA), bits), mx.scale_codes(amax * (1 + DELTA), bits)
    assert np.all((sc >= lo) & (sc <= hi))
    val = mx.mx_dequantize(q.cpu().numpy(), sc, bits)
    ends = [mx.mx_dequantize(mx.pack(mx.elements(y64 * f, sc, bits), bits), sc, bits)
            for f in (1 - DELTA, 1 + DELTA)]
    assert np.all((val >= np.minimum(*ends)) & (val <= np.maximum(*ends)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,H", [(1, 32), (5, 64), (3, 2080), (7, 4096), (2, 8224), (3, 16384), (1, 32768)])
def test_norm(dtype, bits, T, H):
    x = rnd(T, H, seed=T).to(dtype).cuda()
    res = (rnd(T, H, seed=T + 1) * torch.exp(rnd(H, seed=5))).to(dtype).cuda()
    w = (1 + 0.2 * rnd(H, seed=6)).to(dtype).cuda()
    got = mq.moe_rmsnorm_mx(x, w, eps=1e-5, residual=res, bits=bits, want_y=True)
    done()
    check_norm(x, res, w, 1e-5, bits, got)


def test_norm_options():
    """No residual; float32 weight; strided rows; sums written over the
    residual; outputs given by the caller; no rows."""
    T, H = 19, 576
    x = rnd(T, H + 64, seed=1).to(torch.bfloat16).cuda()[:, :H]
    res = rnd(T, H, seed=2).to(torch.bfloat16).cuda()
    w32 = (1 + 0.2 * rnd(H, seed=3)).cuda()
    got = mq.moe_rmsnorm_mx(x, w32, bits=8)
    assert got[2] is None and got[3] is None
    check_norm(x, None, w32, 1e-6, 8, got)
    wide = rnd(2 * T, H, seed=4).to(torch.bfloat16).cuda()[::2]
    check_norm(x, wide, w32, 1e-6, 4, mq.moe_rmsnorm_mx(x, w32, residual=wide, bits=4, want_y=True))
    before = res.clone()
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    got = mq.moe_rmsnorm_mx(x, w32.to(torch.bfloat16), residual=res, residual_out=res, y=y)
    assert got[2] is res and got[3] is y
    check_norm(x, before, w32.to(torch.bfloat16), 1e-6, 8, got)
    assert mq.moe_rmsnorm_mx(x[:0], w32)[0].shape == (0, H)
    done()


def test_norm_of_zeros_and_infinities():
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    x[2, 5] = float("inf")
    x[3, 64] = float("nan")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    q, s, _, y = mq.moe_rmsnorm_mx(x, w, bits=8, want_y=True)
    done()
    assert not q[0].any() and not s[0].any() and not y[0].any()
    assert torch.isfinite(y[1]).all() and (s[1] != 255).all()
    assert (s[2, 0] == 255) and (s[3] == 255).all()   # inf * 0 in that block; NaN everywhere
    assert not q[3].any()


# ------------------------------------------------------------------- product --
def product_case(R, E, K, N, bits, loads, seed=0):
    a = np64(rnd(R, K, seed=seed)) * np.exp(np64(rnd(K, seed=seed + 1)))
    w = np64(rnd(E, N, K, seed=seed + 2, std=0.05))
    qa, sa = cuda_mx(a, bits)
    qw, sw = cuda_mx(w, 4)
    offs = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)
    av = mx.mx_dequantize(qa.cpu().numpy(), sa.cpu().numpy(), bits)
    wv = mx.mx_dequantize(qw.cpu().numpy(), sw.cpu().numpy(), 4)
    return qa, sa, qw, sw, torch.from_numpy(offs).cuda(), mx.mx_product(av, wv, offs)


def check_product(got, ref, mag, K):
    tol = (K / 32 + 10) * 2.0 ** -22 * mag + HALF_ULP[got.dtype] * np.abs(ref)
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), (err / tol).max()


LOADS = [
    (1, 1, 128, 1, [1]),
    (1, 1, 4096, 256, [1]),
    (5, 1, 256, 33, [5]),
    (7, 3, 384, 130, [3, 0, 4]),
    (70, 4, 512, 64, [0, 70, 0, 0]),
    (200, 5, 640, 257, [1, 97, 96, 2, 4]),
    (300, 2, 768, 128, [17, 283]),
    (40, 40, 1408, 160, [1] * 40),
    (33, 2, 2048, 385, [32, 1]),
    (500, 1, 1152, 300, [500]),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,E,K,N,loads", LOADS)
def test_product(R, E, K, N, loads, bits):
    qa, sa, qw, sw, offs, (ref, mag) = product_case(R, E, K, N, bits, loads)
    for dtype in (torch.bfloat16, torch.float32):
        got = mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs, a_bits=bits, out_dtype=dtype)
        done()
        check_product(got, ref, mag, K)


@pytest.mark.parametrize("bits", [4, 8])
def test_product_dense_and_f16(bits):
    qa, sa, qw, sw, _, (ref, mag) = product_case(19, 1, 896, 200, bits, [19])
    out = torch.empty(19, 200, dtype=torch.float16, device="cuda")
    got = mq.moe_mx_product(qa, sa, qw[0], sw[0], a_bits=bits, out=out)
    done()
    assert got is out
    check_product(got, ref, mag, 896)


@pytest.mark.parametrize("N", [96, 97])
@pytest.mark.parametrize("K", [256, 4096])
def test_product_leaves_rows_outside_alone(K, N):
    qa, sa, qw, sw, _, _ = product_case(20, 2, K, N, 8, [10, 10])
    offs = torch.tensor([3, 9, 15], dtype=torch.int32, device="cuda")
    av = mx.mx_dequantize(qa.cpu().numpy(), sa.cpu().numpy(), 8)
    wv = mx.mx_dequantize(qw.cpu().numpy(), sw.cpu().numpy(), 4)
    ref, mag = mx.mx_product(av, wv, offs.cpu().numpy())
    out = torch.full((20, N), 7.0, dtype=torch.float32, device="cuda")
    mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs, out=out)
    done()
    check_product(out[3:15], ref[3:15], mag[3:15], K)
    assert (out[:3] == 7).all() and (out[15:] == 7).all()


def test_product_bad_offsets_are_flagged():
    """Offsets that fall, or leave [0, R], are kept inside the arrays and
    reported."""
    qa, sa, qw, sw, _, _ = product_case(20, 3, 128, 64, 8, [20, 0, 0])
    for offs in ([0, 12, 5, 20], [-4, 3, 8, 20], [0, 5, 9, 1 << 30]):
        t = torch.tensor(offs, dtype=torch.int32, device="cuda")
        mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=t)
        assert mq.mq_device_status() == mq.MQ_DEV_BAD_OFFSETS
    done()


@pytest.mark.parametrize("bits", [4, 8])
def test_product_nan_scales_stay_in_their_row_and_column(bits):
    qa, sa, qw, sw, offs, (ref, mag) = product_case(12, 1, 256, 160, bits, [12])
    sa[4, 3] = 255
    sw[0, 77, 0] = 255
    got = mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs, a_bits=bits, out_dtype=torch.float32)
    done()
    bad = np.zeros(ref.shape, dtype=bool)
    bad[4], bad[:, 77] = True, True
    assert np.array_equal(np.isnan(np64(got)), bad)
    assert np.all(np.abs(np64(got) - ref)[~bad] <= ((256 / 32 + 10) * 2.0 ** -22 * mag + 2.0 ** -24 * np.abs(ref))[~bad])


@pytest.mark.parametrize("bits", [4, 8])
def test_product_extreme_scales(bits):
    """Scales far from 1 on both sides: products near the ends of float32."""
    qa, sa, qw, sw, offs, _ = product_case(6, 1, 128, 40, bits, [6])
    for ds in (-100, 60):
        s2 = (sa.int() + ds).clamp(0, 254).to(torch.uint8)
        av = mx.mx_dequantize(qa.cpu().numpy(), s2.cpu().numpy(), bits)
        wv = mx.mx_dequantize(qw.cpu().numpy(), sw.cpu().numpy(), 4)
        ref, mag = mx.mx_product(av, wv, offs.cpu().numpy())
        got = mq.moe_mx_product(qa, s2, qw, sw, expert_offsets=offs, a_bits=bits, out_dtype=torch.float32)
        done()
        assert np.all(np.abs(np64(got) - ref) <= 14 * 2.0 ** -22 * mag + 2.0 ** -126)


def test_product_same_result_every_run_and_for_any_row_order():
    qa, sa, qw, sw, offs, _ = product_case(130, 2, 2048, 256, 8, [100, 30])
    first = mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs)
    for _ in range(3):
        assert torch.equal(first, mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs))
    perm = torch.cat([torch.randperm(100), 100 + torch.randperm(30)]).cuda()
    again = mq.moe_mx_product(qa[perm].contiguous(), sa[perm].contiguous(), qw, sw, expert_offsets=offs)
    assert torch.equal(first[perm], again)
    done()


def test_product_on_another_stream():
    qa, sa, qw, sw, offs, (ref, mag) = product_case(33, 1, 512, 128, 8, [33])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs)
    side.synchronize()
    check_product(got, ref, mag, 512)
    done()


# ------------------------------------------------------------------- forward --
def forward_case(T, E, k, H, I, bits, seed=0):
    a = np64(rnd(T, H, seed=seed)) * np.exp(0.5 * np64(rnd(H, seed=seed + 1)))
    qa, sa = cuda_mx(a, bits)
    q13, s13 = cuda_mx(np64(rnd(E, 2 * I, H, seed=seed + 2, std=0.05)), 4)
    q2, s2 = cuda_mx(np64(rnd(E, H, I, seed=seed + 3, std=0.05)), 4)
    top = torch.softmax(rnd(T, E, seed=seed + 4), 1).topk(k, dim=1)
    tw = (top.values / top.values.sum(1, keepdim=True)).cuda()
    return qa, sa, q13, s13, q2, s2, tw, top.indices.to(torch.int32).cuda()


def forward_ref(qa, sa, q13, s13, q2, s2, tw, ids, bits):
    n = lambda t: t.cpu().numpy()  # noqa: E731
    return mx.mx_forward(mx.mx_dequantize(n(qa), n(sa), bits), mx.mx_dequantize(n(q13), n(s13), 4),
                         mx.mx_dequantize(n(q2), n(s2), 4), n(tw), n(ids), bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 128, 256), (16, 8, 2, 128, 256), (37, 5, 3, 384, 640),
                                       (1, 1, 1, 512, 128), (300, 4, 2, 256, 384), (64, 70, 8, 256, 128),
                                       (9, 3, 1, 1408, 1152), (130, 2, 2, 2048, 768)])
def test_forward(T, E, k, H, I, bits):
    c = forward_case(T, E, k, H, I, bits, seed=T)
    got = mq.moe_mx_forward(*c, a_bits=bits)
    done()
    check_forward(np64(got), forward_ref(*c, bits), what=f"mx forward {T} {E} {k} {H} {I} {bits}")


def test_forward_f16_bad_ids_and_workspace():
    c = forward_case(21, 6, 2, 256, 256, 8)
    c[7][3, 0], c[7][5, 1], c[7][9] = -1, 6, 77
    ws = torch.empty(mq.moe_mx_forward_workspace(21, 256, 256, 6, 2, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty(21, 256, dtype=torch.float16, device="cuda")
    got = mq.moe_mx_forward(*c, a_bits=8, out=out, workspace=ws)
    assert mq.mq_device_status() == mq.MQ_DEV_BAD_EXPERT_ID
    ref = forward_ref(*c, 8)
    check_forward(np64(got), ref)
    assert not got[9].any()      # a token whose slots are all left out
    with pytest.raises(mq.MoeqError) as e:
        mq.moe_mx_forward(*c, a_bits=8, workspace=ws[:64])
    assert e.value.status == 4


def test_forward_empty_batch_determinism_and_graph():
    c = forward_case(24, 8, 2, 256, 256, 4)
    empty = [t[:0] if i in (0, 1, 6, 7) else t for i, t in enumerate(c)]
    assert mq.moe_mx_forward(*empty, a_bits=4).shape == (0, 256)
    first = mq.moe_mx_forward(*c, a_bits=4)
    assert torch.equal(first, mq.moe_mx_forward(*c, a_bits=4))
    ws = torch.empty(mq.moe_mx_forward_workspace(24, 256, 256, 8, 2, 4), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.moe_mx_forward(*c, a_bits=4, out=out, workspace=ws)
    g.replay()
    done()
    assert torch.equal(first, out)


def test_norm_route_forward_chain():
    """The block as it is used: residual + norm, router on the 16-bit rows,
    experts on the MX rows."""
    T, H, E, k, I = 48, 512, 8, 2, 384
    x, res = rnd(T, H, seed=1).to(torch.bfloat16).cuda(), rnd(T, H, seed=2).to(torch.bfloat16).cuda()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    gate = rnd(E, H, seed=3, std=0.05).to(torch.bfloat16).cuda()
    w13, s13 = mq.moe_quantize_mx(rnd(E, 2 * I, H, seed=4, std=0.05).to(torch.bfloat16).cuda(), bits=4)
    w2, s2 = mq.moe_quantize_mx(rnd(E, H, I, seed=5, std=0.05).to(torch.bfloat16).cuda(), bits=4)
    q, s, h, y = mq.moe_rmsnorm_mx(x, w, residual=res, bits=8, want_y=True)
    tw, ids = mq.moe_topk_route((y @ gate.T).float(), k, True)
    out = mq.moe_mx_forward(q, s, w13, s13, w2, s2, tw, ids, a_bits=8)
    done()
    check_norm(x, res, w, 1e-6, 8, (q, s, h, y))
    check_forward(np64(out), forward_ref(q, s, w13, s13, w2, s2, tw, ids, 8))
