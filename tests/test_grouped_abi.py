"""Host-side refusals of the 16-bit operators (no GPU needed: every call fails its
checks before anything is launched), and their formulas' helpers."""

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
TOP = (1 << 31) - 1


def test_product_refusals(lib):
    def p(a=P, st=64, dt=BF16, R=4, K=64, N=72, E=2, w=P, ws=64, we=64 * 72, tr=0, off=P, out=P, odt=BF16, wk=None, nb=0):
        return lib.moe_grouped_product(a, st, dt, R, K, N, E, w, ws, we, tr, off, out, odt, wk, nb, None)
    assert p(dt=3) == 1 and p(dt=F32) == 2 and p(odt=5) == 1 and p(odt=-1) == 1
    assert p(R=-1) == 1 and p(K=0) == 1 and p(N=0) == 1 and p(E=0) == 1
    assert p(E=1025) == 2 and p(R=1 << 30) == 2
    assert p(K=TOP) == 2 and p(N=TOP) == 2 and p(N=TOP - 511, R=1 << 29) == 2
    assert p(off=None) == 1
    assert p(st=56) == 1 and p(st=68) == 1 and p(ws=56) == 1 and p(ws=60) == 1 and p(ws=-64) == 1
    assert p(we=0) == 1 and p(we=-8) == 1 and p(we=68) == 1
    assert p(tr=1) == 1 and p(tr=1, ws=72, a=None) == 1     # a transposed row has N elements
    assert p(a=None) == 1 and p(w=None) == 1 and p(out=None) == 1
    assert p(a=ODD) == 1 and p(w=ODD) == 1 and p(out=ODD) == 1 and p(off=vp(0x1002)) == 1
    assert p(st=1 << 39) == 2 and p(we=1 << 39) == 2 and p(ws=1 << 39) == 2
    assert b"2^39" in lib.mq_last_error_message()
    assert p(R=0, a=None, out=None) == 0
    # one row, one expert: strides that are never taken are not looked at
    assert p(R=1, st=0, a=ODD) == 1 and b"aligned" in lib.mq_last_error_message()
    assert lib.moe_grouped_product_workspace(-1, 64, 64, 1) == 0
    assert lib.moe_grouped_product_workspace(0, 64, 64, 1) == 0
    assert lib.moe_grouped_product_workspace(4, 64, 64, 2000) == 0
    need = lib.moe_grouped_product_workspace(1, 4096, 256, 1)
    assert need > 0
    for wk, nb in ((None, 0), (P, need - 1), (None, need)):
        assert p(R=1, K=4096, N=256, E=1, st=4096, ws=4096, off=None, wk=wk, nb=nb) == 4
    assert p(R=1, K=4096, N=256, E=1, st=4096, ws=4096, off=None, wk=ODD, nb=need) == 1


def test_gradient_refusals(lib):
    def g(dy=P, dst=72, a=P, ast=64, dt=BF16, R=4, K=64, N=72, E=2, w=P, ws=64, we=64 * 72, tr=0, off=P, da=P, dw=P,
          wdt=F32, wk=None, nb=0):
        return lib.moe_grouped_product_grad(dy, dst, a, ast, dt, R, K, N, E, w, ws, we, tr, off, da, dw, wdt, wk, nb, None)
    assert g(dt=F32) == 2 and g(dt=4) == 1 and g(wdt=3) == 1
    assert g(dst=64) == 1 and g(dst=76) == 1 and g(ast=56) == 1 and g(ast=66) == 1
    assert g(ws=56) == 1 and g(we=0) == 1 and g(off=None) == 1
    assert g(dy=None) == 1 and g(a=None) == 1 and g(w=None) == 1
    for k in ("dy", "a", "w", "da", "dw"):
        assert g(**{k: ODD}) == 1, k
    assert g(da=None, dw=None) == 0                       # nothing asked for
    assert g(dw=None, a=None, w=None) == 1                # the rows' gradient reads w ...
    assert g(da=None, w=None, ws=0, we=0, a=None) == 1    # ... the weights' reads a
    assert g(R=0, dw=None) == 0
    assert g(R=-1) == 1 and g(E=1025) == 2 and g(K=TOP) == 2 and g(N=TOP) == 2
    assert lib.moe_grouped_product_grad_workspace(4, 0, 64, 2) == 0
    need = lib.moe_grouped_product_grad_workspace(4096, 64, 64, 1)
    assert need > 0
    assert g(R=4096, N=64, E=1, dst=64, nb=need, wk=None) == 4
    assert g(R=4096, N=64, E=1, dst=64, nb=need - 1, wk=P) == 4


def test_binding_refusals(lib):
    """Wrong dtypes, devices, shapes and strides never reach the library."""
    from weight_quantized_moe_gb300 import binding as b
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        b.moe_grouped_product(x, w)
    with pytest.raises(TypeError):
        b.moe_grouped_product(x.float(), w)
    with pytest.raises(TypeError):
        b.moe_grouped_product(x, w, out_dtype=torch.int32)
    with pytest.raises(TypeError):
        b.moe_grouped_product([1.0], w)
    with pytest.raises(TypeError):
        b.moe_grouped_product_grad(x, x, w, dw_dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        b.moe_grouped_product_grad(x, x, w)


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from grouped_fake_device import compile_fake
    return compile_fake(str(tmp_path_factory.mktemp("grouped_fake")))


@pytest.fixture
def on(fake):
    keep = []   # host memory behind the tensors

    def make(t, device=0):
        keep.append(t)
        return fake[1].on_device(t, device)
    fake[1].calls()
    return make


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_compiled_calls_check_shapes_and_strides(fake, on):
    calls, pretend = fake
    a, w, off = on(z(4, 64)), on(z(2, 8, 64)), on(z(3, dtype=torch.int32))

    def refused(match, *args, call=calls.product, kind=ValueError):
        with pytest.raises(kind, match=match):
            call(*args)
    ok = (a, w, off, None, 0, None)
    refused("length", on(z(4, 72)), *ok[1:])
    refused("E \\+ 1", a, w, on(z(2, dtype=torch.int32)), *ok[3:])
    refused("Int", a, w, on(z(3, dtype=torch.int64)), *ok[3:], kind=TypeError)
    refused("missing", a, w, None, *ok[3:])
    refused("2 dims", on(z(64)), *ok[1:])
    refused("2 or 3 dims", a, on(z(1, 2, 8, 64)), *ok[2:])
    refused("BFloat16", a, on(z(2, 8, 64, dtype=torch.float16)), *ok[2:], kind=TypeError)
    refused("cuda:0", a, on(z(2, 8, 64), 1), *ok[2:])
    refused("cuda:0", a, w, on(z(3, dtype=torch.int32), 1), *ok[3:])
    refused("contiguous", on(z(64, 4).T), *ok[1:])
    refused("contiguous rows", a, on(z(2, 8, 128)[:, :, ::2]), *ok[2:])
    refused("shape", *ok[:3], on(z(4, 9)), *ok[4:])
    refused("Float", *ok[:3], on(z(4, 8)), 2, None, kind=TypeError)
    refused("least one element", on(z(4, 0)), on(z(2, 8, 0)), *ok[2:])
    refused("empty", a, on(z(0, 8, 64)), *ok[2:])
    grad = (on(z(4, 8)), a, w, off, True, True, on(z(4, 64)), None, 0, None)
    refused("dy must be", on(z(3, 8)), *grad[1:], call=calls.product_grad)
    refused("dy must be", on(z(4, 16)), *grad[1:], call=calls.product_grad)
    refused("w's shape", *grad[:7], on(z(2, 64, 8)), 0, None, call=calls.product_grad)
    refused("order", *grad[:7], on(z(2, 64, 8).transpose(1, 2)), 0, None, call=calls.product_grad)
    assert pretend.calls() == ([], 0)


@pytest.mark.parametrize("device", [0, 1, 3])
def test_compiled_calls_launch_on_their_tensors_device(fake, on, device):
    calls, pretend = fake
    t = lambda *s, **k: on(z(*s, **k), device)  # noqa: E731
    off, ws = t(3, dtype=torch.int32), t(16, dtype=torch.uint8)
    calls.product(t(4, 64), t(2, 8, 64), off, t(4, 8), 0, ws)
    calls.product_grad(t(4, 8), t(4, 64), t(2, 8, 64), off, True, True, t(4, 64), t(2, 8, 64), 0, ws)
    assert pretend.calls() == ([(device, 100 + device)] * 2, 0)


def test_weights_storage(fake, on):
    """(row stride, expert stride, transposed) that the library gets."""
    calls, pretend = fake
    off = on(z(3, dtype=torch.int32))

    def of(w, out=None):
        K, N = w.shape[-1], w.shape[-2]
        a = on(z(4, -(-K // 8) * 8)[:, :K])
        calls.product(a, on(w), off if w.dim() == 3 and w.shape[0] == 2 else None, on(z(4, N)), 0, None)
        return pretend.weights()
    assert of(z(2, 8, 64)) == (64, 512, 0)
    assert of(z(2, 64, 8).transpose(1, 2)) == (8, 512, 1)
    assert of(z(2, 16, 128)[:, 8:, 64:]) == (128, 2048, 0)
    assert of(z(8, 2, 64).transpose(0, 1)) == (128, 64, 0)
    assert of(z(8, 64))[::2] == (64, 0)
    assert of(z(64, 8).T)[::2] == (8, 1)
    assert of(z(1, 64))[::2] == (64, 0)       # one row: its stride is never taken
    assert of(z(33, 1))[2] == 1               # one column: a row of the other storage
    assert of(z(2, 8, 40)[:, :, :33])[::2] == (40, 0)
