"""Host-side refusals of the microscaled operators (no GPU needed: every call
fails its checks before anything is launched)."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from weight_quantized_moe_gb300 import binding, build
    build.build()
    return binding.lib()


vp = ctypes.c_void_p
P = vp(0x1000)       # never dereferenced
ODD = vp(0x1008)     # not 16-byte aligned
BF16, F16, F32 = 0, 1, 2


def test_quantize_mx_refusals(lib):
    q = lambda x=P, dt=BF16, rows=4, cols=64, st=64, bits=4, c=P, s=P: lib.moe_quantize_mx(  # noqa: E731
        x, dt, rows, cols, st, bits, c, s, None)
    assert q(dt=3) == 1 and q(dt=-1) == 1
    assert q(bits=6) == 1
    assert q(rows=-1) == 1
    assert q(cols=0) == 1 and q(cols=48) == 1
    assert q(st=32) == 1 and q(st=68) == 1
    assert q(x=None) == 1 and q(c=None) == 1 and q(s=None) == 1
    assert q(x=ODD) == 1 and q(c=ODD) == 1 and q(s=vp(0x1002)) == 1
    assert q(rows=1 << 36, cols=64) == 2
    assert q(rows=0, x=None, c=None, s=None) == 0
    d = lambda **k: lib.moe_dequantize_mx(k.get("c", P), k.get("s", P), k.get("rows", 4),  # noqa: E731
                                          k.get("cols", 64), k.get("bits", 8), k.get("out", P),
                                          k.get("dt", F32), None)
    assert d(cols=40) == 1 and d(bits=5) == 1 and d(dt=7) == 1 and d(out=ODD) == 1 and d(c=None) == 1
    assert d(rows=0, out=None, c=None, s=None) == 0


def test_rmsnorm_mx_refusals(lib):
    def n(x=P, res=None, w=P, dt=BF16, T=4, H=64, xs=64, rs=64, eps=1e-6, ro=None, y=None, bits=8, q=P, s=P):
        return lib.moe_rmsnorm_mx(x, res, w, dt, 0, T, H, xs, rs, eps, ro, y, bits, q, s, None)
    assert n(dt=F32) == 2 and n(dt=9) == 1
    assert n(H=40) == 1 and n(H=0) == 1 and n(H=32800, xs=32800) == 2
    assert n(T=-1) == 1 and n(T=0, x=None) == 0
    assert n(xs=32) == 1 and n(xs=66) == 1 and n(res=P, rs=60) == 1
    assert n(eps=-1.0) == 1 and n(eps=float("nan")) == 1 and n(eps=float("inf")) == 1
    assert n(bits=3) == 1
    assert n(x=None) == 1 and n(w=None) == 1 and n(q=None) == 1 and n(s=None) == 1
    assert n(x=ODD) == 1 and n(y=ODD) == 1 and n(ro=ODD) == 1 and n(w=ODD) == 1
    other = vp(0x9000)
    assert n(x=other, res=P, rs=128, ro=P) == 1      # in place needs a dense residual
    assert b"dense" in lib.mq_last_error_message()


def test_mx_product_refusals(lib):
    def p(a=P, s=P, bits=8, R=4, K=128, N=64, E=2, w=P, ws=P, off=P, out=P, dt=BF16, wk=None, nb=0):
        return lib.moe_mx_product(a, s, bits, R, K, N, E, w, ws, off, out, dt, wk, nb, None)
    assert p(bits=16) == 1 and p(dt=4) == 1
    assert p(R=-1) == 1 and p(K=0) == 1 and p(N=0) == 1 and p(E=0) == 1
    assert p(K=160) == 2 and p(E=1025) == 2 and p(R=1 << 30) == 2
    assert p(off=None) == 1
    assert p(R=0, a=None, off=None, E=1) == 0
    assert p(a=None) == 1 and p(w=None) == 1 and p(out=None) == 1
    assert p(w=vp(0x1010)) == 1 and p(a=ODD) == 1 and p(off=vp(0x1002)) == 1
    assert lib.moe_mx_product_workspace(-1, 128, 64, 2) == 0
    assert lib.moe_mx_product_workspace(4, 100, 64, 2) == 0
    need = lib.moe_mx_product_workspace(1, 4096, 4096, 1)
    if need:
        assert p(R=1, K=4096, N=4096, E=1, off=None) == 4
        assert p(R=1, K=4096, N=4096, E=1, off=None, wk=P, nb=need - 1) == 4


def test_mx_forward_refusals(lib):
    def f(a=P, bits=8, T=4, H=128, I=128, E=8, k=2, w13=P, ids=P, out=P, dt=BF16, wk=P, nb=1 << 30):
        return lib.moe_mx_forward(a, P, bits, T, H, I, E, k, w13, P, P, P, P, ids, out, dt, wk, nb, None)
    assert f(bits=5) == 1 and f(dt=F32) == 1
    assert f(T=-1) == 1 and f(H=0) == 1 and f(k=0) == 1 and f(k=9) == 1 and f(E=64, k=33) == 1
    assert f(H=192) == 2 and f(I=100) == 2 and f(E=2000) == 2 and f(T=1 << 24, k=2) == 2
    assert f(a=None) == 1 and f(out=None) == 1 and f(wk=None) == 1
    assert f(w13=vp(0x1010)) == 1 and f(out=ODD) == 1 and f(ids=vp(0x1001)) == 1
    assert f(nb=64) == 4
    assert f(T=0, a=None) == 0
    assert lib.moe_mx_forward_workspace(4, 128, 128, 8, 2, 8) > lib.moe_mx_forward_workspace(4, 128, 128, 8, 2, 4) > 0
    assert lib.moe_mx_forward_workspace(4, 128, 128, 8, 9, 8) == 0
    assert lib.moe_mx_forward_workspace(4, 128, 128, 8, 2, 6) == 0


def test_binding_refusals(lib):
    """Wrong dtypes, devices, shapes and strides never reach the library."""
    from weight_quantized_moe_gb300 import binding as b
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        b.moe_quantize_mx(x)
    with pytest.raises(TypeError):
        b.moe_quantize_mx(x.double())
    with pytest.raises(TypeError):
        b.moe_dequantize_mx(x, x, dtype=torch.int8)
    with pytest.raises(TypeError):
        b.moe_rmsnorm_mx(x.float(), x)
    with pytest.raises(TypeError):
        b.moe_mx_product(x, x, x, x, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        b.moe_mx_forward(x, x, x, x, x, x, x, x, out_dtype=torch.float32)
    with pytest.raises(TypeError):
        b.moe_quantize_mx([1.0])


def test_rmsnorm_mx_outputs_may_not_share_memory_with_other_rows(lib):
    """A row's output over another row's input is written while that row may not
    have been read: refused, for both outputs and both inputs."""
    base = 0x100000
    T, H = 4, 64
    row = 2 * H     # bytes

    def refused(**k):
        rc = n_checked(**k)
        return rc == 1 and b"share" in lib.mq_last_error_message()

    def n_checked(x=base, res=None, ro=None, y=None, xs=H, rs=H, T=T):
        p = lambda v: None if v is None else vp(v)  # noqa: E731
        # (the weight is misaligned: a call whose rows pass is refused for that)
        return lib.moe_rmsnorm_mx(p(x), p(res), ODD, BF16, 0, T, H, xs, rs, 1e-6, p(ro), p(y), 8, P, P, None)
    far = base + 0x80000
    for out in ("y", "ro"):
        assert refused(**{out: base, "xs": 2 * H})                     # dense rows over strided ones
        assert refused(**{out: base + row})                            # the same rows, one on
        assert refused(**{out: base - row})
        assert refused(**{out: base + 16, "xs": 2 * H})                # across a gap
        assert refused(x=far, res=base, **{out: base, "rs": H + 64})
        assert refused(x=far, res=base, **{out: base + (T - 1) * row})
        # in place, between the rows, before and behind them: not refused for this
        assert not refused(**{out: base})
        assert not refused(x=far, res=base, **{out: base})
        assert not refused(**{out: base + T * row})
        assert not refused(**{out: base - T * row})
        assert not refused(**{out: base + row, "xs": (T + 1) * H})     # all of it in one gap
        assert refused(**{out: base + row + 16, "xs": (T + 1) * H})
        assert not refused(**{out: base, "xs": 2 * H, "T": 1})         # a single row has no stride
    assert refused(y=base + row, ro=base, x=far)                       # the outputs on one another
    assert not refused(y=base + T * row, ro=base, x=far)


def test_quantize_mx_strided_rows_past_the_kernels_row_count_are_refused(lib):
    """Strided rows are found by dividing by the row's vectors of eight, counted in
    32 bits; rows of 2^35 elements have more.  (Refused before anything is
    launched; dense ones need no division.)"""
    def q(cols, st, rows=2, x=P):
        # (the scale is misaligned: a call whose sizes pass is refused for that)
        rc = lib.moe_quantize_mx(x, BF16, rows, cols, st, 4, P, vp(0x1002), None)
        return rc
    assert q(1 << 35, (1 << 35) + 8) == 2
    assert q(1 << 36, 1 << 37, rows=1) == 2
    assert b"dense" in lib.mq_last_error_message()
    assert q(1 << 35, 1 << 35) == 1
    assert q((1 << 35) - 32, 1 << 35) == 1


def test_mx_sizes_whose_rounded_up_values_pass_32_bits_are_refused(lib):
    """The product counts weight rows in tiles of 256 past its last one, k in
    steps of 512; a forward has 2I weight rows and rows of H * a_bits bits."""
    top = (1 << 31) - 1

    # (a is misaligned: a call whose sizes pass is refused for that)
    def p(K=128, N=64):
        return lib.moe_mx_product(ODD, P, 8, 1, K, N, 1, P, P, None, P, BF16, None, 0, None)
    assert p(N=top) == 2 and p(N=top - 510) == 2 and p(N=top - 511) == 1
    assert p(K=(1 << 31) - 128) == 2 and p(K=(1 << 31) - 384) == 2 and p(K=(1 << 31) - 512) == 1
    for K, N in ((128, top), ((1 << 31) - 128, 64)):
        assert lib.moe_mx_product_workspace(1, K, N, 1) == 0

    def f(H=128, I=128, bits=8, T=1):
        return lib.moe_mx_forward(ODD, P, bits, T, H, I, 1, 1, P, P, P, P, P, P, P, BF16, P, 1 << 62, None)
    assert f(I=1 << 30) == 2 and f(I=(1 << 30) + 128) == 2 and f(I=(1 << 31) - 128) == 2
    assert f(H=1 << 28) == 2 and f(H=(1 << 31) - 128) == 2
    assert f(I=(1 << 30) - 128) == 2 and f(I=(1 << 30) - 256) == 1 and f(H=(1 << 28) - 128) == 1


def test_mx_forward_workspace_is_0_for_sizes_that_the_forward_refuses(lib):
    """Else a caller allocates, or fails to, before it is told."""
    w = lib.moe_mx_forward_workspace

    def refused(T=4, H=128, I=128, E=8, k=2, bits=8):
        assert lib.moe_mx_forward(P, P, bits, T, H, I, E, k, P, P, P, P, P, P, P, BF16, vp(0x1001), 1 << 62,
                                  None) in (1, 2)
        return w(T, H, I, E, k, bits) == 0
    assert w(4, 128, 128, 8, 2, 8) > 0
    assert refused(E=64, k=33) and refused(E=1025) and refused(H=192) and refused(I=100)
    assert refused(T=1 << 24, k=2) and refused(T=(1 << 31) - 1, E=64, k=32)
    assert refused(I=1 << 30) and refused(H=1 << 28) and refused(T=-1)
    assert refused(T=1 << 20, H=1 << 24, I=1 << 24)      # too many units of work
