"""Where the microscaled operators can go wrong: sizes that only the largest
inputs reach, chunk and tile borders of both kernel shapes, other streams,
non-finite rows, lopsided loads, refusals.  Tolerances as derived in
test_gpu_mx.py."""

import numpy as np
import pytest
import torch

from moe_helpers import check_forward
from oracle import mx_oracle as mx
from test_gpu_mx import (HALF_ULP, check_product, cuda_mx, done, forward_case, forward_ref, np64,
                         product_case, rnd)

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("weight_quantized_moe_gb300")


# ------------------------------------------------- chunk and tile borders ----
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,E,K,N,loads", [
    (97, 1, 128, 1, [97]),                  # the first size of the paired kernel
    (224, 1, 256, 255, [224]),              # exactly one of its chunks
    (225, 1, 640, 257, [225]),              # one row more, one output more than its tile
    (448, 2, 1280, 512, [0, 448]),          # an empty expert first
    (700, 3, 384, 129, [31, 33, 636]),      # chunks of 31, 33 and 188 rows
    (96, 1, 512, 300, [96]),                # the last size of the single kernel
    (64, 2, 128, 700, [16, 48]),
    (33, 33, 896, 96, [1] * 33),
    (41, 2, 3200, 513, [41, 0]),
])
def test_product_borders(R, E, K, N, loads, bits):
    qa, sa, qw, sw, offs, (ref, mag) = product_case(R, E, K, N, bits, loads, seed=R)
    got = mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs, a_bits=bits, out_dtype=torch.float32)
    done()
    check_product(got, ref, mag, K)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,E,k,H,I", [(200, 2, 1, 256, 128), (333, 3, 3, 128, 640), (225, 1, 1, 384, 256),
                                       (97, 1, 1, 128, 384), (450, 4, 2, 640, 384)])
def test_forward_borders(T, E, k, H, I, bits):
    c = forward_case(T, E, k, H, I, bits, seed=T + 7)
    got = mq.moe_mx_forward(*c, a_bits=bits)
    done()
    check_forward(np64(got), forward_ref(*c, bits), what=f"mx forward {T} {E} {k} {H} {I} {bits}")


@pytest.mark.parametrize("T", [20, 400])
def test_forward_all_tokens_on_one_expert(T):
    c = forward_case(T, 64, 1, 256, 256, 8, seed=3)
    c[7].fill_(63)
    got = mq.moe_mx_forward(*c, a_bits=8)
    done()
    check_forward(np64(got), forward_ref(*c, 8))


# ------------------------------------------------------------- large inputs --
def test_product_long_unit_lists_and_output_past_32_bits():
    """Over 2^31 outputs, and more units per CTA than its list holds; sampled
    rows against 64 bits."""
    R, K, N = 80000, 128, 28672
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(R, K, generator=g, device="cuda")
    w = torch.randn(N, K, generator=g, device="cuda") * 0.1
    qa, sa = mq.moe_quantize_mx(a, bits=8)
    qw, sw = mq.moe_quantize_mx(w, bits=4)
    out = mq.moe_mx_product(qa, sa, qw, sw, a_bits=8)
    done()
    wv = mx.mx_dequantize(qw.cpu().numpy(), sw.cpu().numpy(), 4)
    rows = torch.tensor([0, 1, 223, 224, 40000, 74898, 74899, R - 2, R - 1])
    av = mx.mx_dequantize(qa[rows.cuda()].cpu().numpy(), sa[rows.cuda()].cpu().numpy(), 8)
    check_product(out[rows.cuda()], av @ wv.T, np.abs(av) @ np.abs(wv).T, K)


def test_product_many_experts_long_unit_lists():
    """1024 experts of a row or two: over 128 units per CTA of the single kernel."""
    E, K, N = 1024, 128, 6400
    g = torch.Generator(device="cuda").manual_seed(2)
    loads = torch.tensor([1, 2] * (E // 2))
    offs = torch.cat([torch.zeros(1, dtype=torch.int64), loads.cumsum(0)]).to(torch.int32)
    R = int(offs[-1])
    qa, sa = mq.moe_quantize_mx(torch.randn(R, K, generator=g, device="cuda"), bits=4)
    qw = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sw = torch.randint(118, 124, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    out = mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs.cuda(), a_bits=4)
    done()
    av = mx.mx_dequantize(qa.cpu().numpy(), sa.cpu().numpy(), 4)
    for e in (0, 1, 511, 777, 1022, 1023):
        wv = mx.mx_dequantize(qw[e].cpu().numpy(), sw[e].cpu().numpy(), 4)
        s = slice(int(offs[e]), int(offs[e + 1]))
        check_product(out[s], av[s] @ wv.T, np.abs(av[s]) @ np.abs(wv).T, K)


def test_quantise_past_32_bits():
    rows, cols = 300000, 8192          # 2.46e9 elements
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 131071, 262143, 262144, 262145, rows - 1])
    x[at.cuda()] = rnd(len(at), cols, seed=4).to(torch.bfloat16).cuda()
    q, s = mq.moe_quantize_mx(x, bits=4)
    v = mq.moe_dequantize_mx(q, s, bits=4)
    done()
    oq, os_ = mx.mx_quantize(np64(x[at.cuda()]), 4)
    assert np.array_equal(q[at.cuda()].cpu().numpy(), oq)
    assert np.array_equal(s[at.cuda()].cpu().numpy(), os_)
    assert np.array_equal(np64(v[at.cuda()]), mx.mx_dequantize(oq, os_, 4))
    assert not v[1].any() and not v[rows - 2].any()


# ------------------------------------------------------------------ streams --
def test_calls_on_a_given_stream():
    """stream=: inputs made on that stream, workspaces reused call after call."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = rnd(48, 512, seed=1).to(torch.bfloat16).cuda(non_blocking=True)
        w = rnd(300, 512, seed=2, std=0.05).cuda(non_blocking=True)
    q, s = mq.moe_quantize_mx(x, bits=8, stream=side)
    qw, sw = mq.moe_quantize_mx(w, bits=4, stream=side)
    outs = [mq.moe_mx_product(q, s, qw, sw, a_bits=8, stream=side) for _ in range(8)]
    side.synchronize()
    av = mx.mx_dequantize(*mx.mx_quantize(np64(x), 8), 8)
    wv = mx.mx_dequantize(*mx.mx_quantize(np64(w), 4), 4)
    for out in outs:
        check_product(out, av @ wv.T, np.abs(av) @ np.abs(wv).T, 512)


def test_two_streams_at_once():
    cs = [forward_case(40 + 3 * i, 8, 2, 256, 384, 8, seed=i) for i in range(2)]
    refs = [forward_ref(*c, 8) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    for _ in range(6):
        for i, st in enumerate(streams):
            outs[i].append(mq.moe_mx_forward(*cs[i], a_bits=8, stream=st))
    done()
    for i in range(2):
        for out in outs[i]:
            check_forward(np64(out), refs[i])


# ---------------------------------------------------------------- non-finite --
@pytest.mark.parametrize("T", [12, 260])
def test_forward_non_finite_token_stays_alone(T):
    c = forward_case(T, 2, 2, 256, 256, 8, seed=5)
    c[1][3, 0] = 255                   # a NaN block of one token
    got = np64(mq.moe_mx_forward(*c, a_bits=8))
    done()
    assert np.isnan(got[3]).all() and np.isfinite(np.delete(got, 3, 0)).all()
    ref = forward_ref(*[t[[i for i in range(T) if i != 3]].contiguous() if j in (0, 1, 6, 7) else t
                        for j, t in enumerate(c)], 8)
    check_forward(np.delete(got, 3, 0), ref)


@pytest.mark.parametrize("T", [10, 250])
def test_forward_saturated_gates(T):
    """Gate values far below and above the range of exp."""
    c = forward_case(T, 2, 1, 256, 256, 8, seed=8)
    c[1].add_(8)                       # rows 256 times as large: |gate| of some hundreds
    ref = forward_ref(*c, 8)
    got = mq.moe_mx_forward(*c, a_bits=8)
    done()
    assert np.isfinite(ref).all()
    check_forward(np64(got), ref)


def test_forward_of_zero_tokens_rows():
    """Rows of zeros: every block scale is the smallest, the output is 0."""
    c = forward_case(9, 4, 2, 256, 256, 4, seed=6)
    c[0].zero_()
    c[1].zero_()
    got = mq.moe_mx_forward(*c, a_bits=4)
    done()
    assert not got.any()


# ------------------------------------------------------------------ refusals --
def test_python_refusals():
    qa, sa = cuda_mx(np.ones((4, 256)), 8)
    qw, sw = cuda_mx(np.ones((2, 96, 256)), 4)
    offs = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    ok = dict(expert_offsets=offs, a_bits=8)
    assert mq.moe_mx_product(qa, sa, qw, sw, **ok).shape == (4, 96)
    for bad in (
        lambda: mq.moe_mx_product(qa, sa[:3], qw, sw, **ok),
        lambda: mq.moe_mx_product(qa, sa, qw, sw, a_bits=8),              # experts without offsets
        lambda: mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs[:2], a_bits=8),
        lambda: mq.moe_mx_product(qa, sa, qw, sw, expert_offsets=offs.long(), a_bits=8),
        lambda: mq.moe_mx_product(qa[:, :128], sa[:, :4], qw, sw, **ok),   # strided rows
        lambda: mq.moe_mx_product(qa, sa, qw.cpu(), sw.cpu(), **ok),
        lambda: mq.moe_mx_product(qa, sa, qw, sw, out=torch.empty(4, 95, device="cuda"), **ok),
        lambda: mq.moe_mx_product(qa, sa, qw, sw, out_dtype=torch.float64, **ok),
        lambda: mq.moe_mx_product(qa, sa.float(), qw, sw, **ok),
        lambda: mq.moe_mx_product(None, sa, qw, sw, **ok),
        lambda: mq.moe_quantize_mx(torch.ones(4, 40, device="cuda")),
        lambda: mq.moe_quantize_mx(torch.ones(4, 64, device="cuda")[:, ::2]),
        lambda: mq.moe_quantize_mx(torch.ones(4, 64, device="cuda"), bits=2),
        lambda: mq.moe_quantize_mx(torch.ones(4, 64, device="cuda", dtype=torch.int32)),
        lambda: mq.moe_dequantize_mx(qa, sa, bits=4),
        lambda: mq.moe_rmsnorm_mx(torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")),
        lambda: mq.moe_rmsnorm_mx(torch.ones(4, 64, device="cuda").half(), torch.ones(32, device="cuda")),
        lambda: mq.moe_rmsnorm_mx(torch.ones(4, 64, device="cuda").half(), torch.ones(64, device="cuda"),
                                  residual=torch.ones(4, 64, device="cuda")),
    ):
        with pytest.raises((TypeError, ValueError, mq.MoeqError)):
            bad()
    done()


def test_norm_row_strides_that_the_kernel_cannot_read_are_refused():
    wide = torch.ones(4, 100, device="cuda").half()
    with pytest.raises(mq.MoeqError):      # rows 100 elements apart: not 16-byte aligned
        mq.moe_rmsnorm_mx(wide[:, :64], torch.ones(64, device="cuda").half())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_product_output_rounding_is_one_rounding(dtype):
    """Exact integers: the result is the exact sum, rounded once."""
    a = np.tile(np.array([1.0, 2, 3, 4, -1, -2, 6, 0.5]), (5, 32))
    w = np.tile(np.array([1.0, 0.5, -1, 2, 1, 4, 1, 6]), (40, 32))
    qa, sa = cuda_mx(a, 4)
    qw, sw = cuda_mx(w, 4)
    got = mq.moe_mx_product(qa, sa, qw, sw, a_bits=4, out_dtype=dtype)
    done()
    av, wv = mx.mx_dequantize(*mx.mx_quantize(a, 4), 4), mx.mx_dequantize(*mx.mx_quantize(w, 4), 4)
    want = torch.from_numpy(av @ wv.T).float().to(dtype)
    assert torch.equal(got.cpu(), want)
    assert HALF_ULP[dtype] > 0
