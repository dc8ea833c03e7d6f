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
    # (one row times weights stored [E, K, N] is summed in splits; stored [E, N, K] it needs no workspace)
    for wk, nb in ((None, 0), (P, need - 1), (None, need)):
        assert p(R=1, K=4096, N=256, E=1, st=4096, ws=256, tr=1, off=None, wk=wk, nb=nb) == 4
    assert p(R=1, K=4096, N=256, E=1, st=4096, ws=256, tr=1, off=None, wk=ODD, nb=need) == 1


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


def test_product_and_gradients_share_no_memory_with_their_inputs(lib):
    """Results on top of an input, or ending or beginning inside one (no workspace is needed)."""
    R, K, N, E = 64, 64, 128, 8
    A, W, OFF, Y, DA, DW = (vp(0x1000000 * i) for i in range(1, 7))
    sizes = {"a": 2 * R * K, "w": 2 * E * N * K, "off": 4 * (E + 1), "dy": 2 * R * N}

    def product(out, transposed=0, a_stride=K):
        rc = lib.moe_grouped_product(A, a_stride, BF16, R, K, N, E, W, N if transposed else K, N * K, transposed, OFF,
                                     out, BF16, None, 0, None)
        return rc == 1 and b"share" in lib.mq_last_error_message()
    assert lib.moe_grouped_product_workspace(R, K, N, E) == 0

    def grad(da, dw):
        rc = lib.moe_grouped_product_grad(Y, N, A, K, BF16, R, K, N, E, W, K, N * K, 0, OFF, da, dw, F32, P,
                                          1 << 40, None)
        return rc == 1 and b"share" in lib.mq_last_error_message()
    out, da, dw = 2 * R * N, 2 * R * K, 4 * E * N * K
    for name, at in (("a", A), ("w", W), ("off", OFF)):
        for t in (0, 1):
            assert product(at, t) and product(vp(at.value + sizes[name] // 16 * 16 - 16), t), name
            assert product(vp(at.value - out + 16), t), name
    assert product(vp(A.value + 2 * (R - 1) * 1024 + 2 * K - 16), a_stride=1024)
    for name, at in (("a", A), ("w", W), ("off", OFF), ("dy", Y)):
        for place in (at.value, at.value + sizes[name] // 16 * 16 - 16):
            assert grad(vp(place), DW) and grad(DA, vp(place)), name
        assert grad(vp(at.value - da + 16), DW) and grad(DA, vp(at.value - dw + 16)), name
    assert grad(DA, DA) and grad(DA, vp(DA.value + da - 16)) and grad(vp(DW.value + dw - 16), DW)


def test_lora_refusals(lib):
    far, farther = vp(0x10000000), vp(0x20000000)

    def q(x=P, st=64, dt=BF16, R=4, K=64, N=72, r=16, L=3, E=2, a=P, b=P, ids=P, off=P, sc=None, base=far, bs=72,
          out=farther, os=72, odt=BF16, wk=None, nb=0):
        return lib.moe_lora_product(x, st, dt, R, K, N, r, L, E, a, b, ids, off, sc, base, bs, out, os, odt, wk, nb, None)
    # (the scaling is misaligned: a call that passes the checks before it is refused for that)
    last = dict(sc=vp(0x1002))
    assert q(**last) == 1 and b"aligned" in lib.mq_last_error_message()
    assert q(dt=F32) == 2 and q(dt=3) == 1 and q(odt=7) == 1
    assert q(R=-1) == 1 and q(K=0) == 1 and q(N=0) == 1 and q(r=0) == 1 and q(L=0) == 1 and q(E=0) == 1
    assert q(K=68, st=72) == 1 and q(r=12) == 1
    assert q(r=136) == 2 and q(E=1025) == 2 and q(R=1 << 30) == 2 and q(K=1 << 30, st=1 << 30) == 2
    assert q(N=1 << 30) == 2 and q(L=1 << 29, E=2) == 2 and q(L=1 << 20, E=512, K=1 << 20, st=1 << 20) == 2
    assert q(off=None) == 1
    assert q(st=56) == 1 and q(st=68) == 1 and q(os=71) == 1 and q(bs=64) == 1
    for k in ("x", "a", "b", "ids", "out"):
        assert q(**{k: None}) == 1, k
    assert q(x=ODD) == 1 and q(a=ODD) == 1 and q(b=ODD) == 1 and q(ids=vp(0x1002)) == 1 and q(off=vp(0x1001)) == 1
    assert q(out=vp(0x20000001)) == 1 and q(base=vp(0x10000001)) == 1 and q(out=vp(0x20000002), odt=F32) == 1
    assert q(st=1 << 39) == 2 and q(os=1 << 39) == 2 and q(bs=1 << 39) == 2
    assert q(R=0, x=None, out=None) == 0
    need = lib.moe_lora_product_workspace(2000, 64, 72, 16, 3, 2)
    assert need > 0
    for wk, nb in ((None, 0), (P, need - 1), (None, need)):
        assert q(R=2000, wk=wk, nb=nb) == 4
    for k, size in (("a", 2 * 3 * 2 * 16 * 64), ("b", 2 * 3 * 2 * 16 * 72), ("ids", 4 * 4), ("off", 4 * 3), ("sc", 4 * 3)):
        for place in (farther, vp(farther.value + 2 * 4 * 72 - 16), vp(farther.value - size // 16 * 16)):
            if place.value < farther.value and size % 16:
                place = vp(farther.value - size + 4)    # its last element is out's first
            elif place.value < farther.value:
                place = vp(place.value + 16) if k in ("a", "b") else vp(place.value + 4)
            assert q(**{k: place}) == 1 and b"share" in lib.mq_last_error_message(), (k, place)
    assert q(R=2000, wk=ODD, nb=need) == 1
    w = lib.moe_lora_product_workspace
    assert w(-1, 64, 72, 16, 3, 2) == 0 and w(0, 64, 72, 16, 3, 2) == 0 and w(2000, 60, 72, 16, 3, 2) == 0
    assert w(2000, 64, 72, 256, 3, 2) == 0


def test_lora_out_may_be_base_but_share_no_other_memory(lib):
    base = 0x1000000
    R, N = 4, 72
    row = 2 * N

    def refused(x=0x9000000, base_=base, bs=N, out=base, os=N, R=R, K=64, st=64):
        # (the workspace is missing: a call whose rows pass is refused for that)
        p = lambda v: None if v is None else vp(v)  # noqa: E731
        rc = lib.moe_lora_product(p(x), st, BF16, R, K, N, 16, 3, 1, P, P, P, None, None, p(base_), bs, p(out), os, BF16,
                                  None, 0, None)
        if rc == 1 and b"share" in lib.mq_last_error_message():
            return True
        assert rc == 4, lib.mq_last_error_message()
        return False
    R = 2000     # (tiles: a workspace is needed)
    k = dict(R=R)
    assert not refused(**k)                                         # in place
    assert not refused(out=base + R * row, **k) and not refused(out=base - R * row, **k)
    assert refused(out=base + row, **k) and refused(out=base - row, **k) and refused(out=base + 2, **k)
    assert refused(out=base + R * row - 2, **k) and refused(bs=80, **k) and refused(os=80, **k)
    # slices of one wider buffer: the rows alternate
    assert not refused(out=base + row, bs=2 * N, os=2 * N, **k)
    assert not refused(out=base - row, bs=2 * N, os=2 * N, **k)
    assert refused(out=base + row - 2, bs=2 * N, os=2 * N, **k)
    assert refused(out=base + row + 2, bs=2 * N, os=2 * N, **k)     # its end reaches base's next row
    assert refused(x=base, **k) and refused(x=base + 16, base_=None, **k)
    assert not refused(base_=None, **k)


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
    ids = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        b.moe_lora_product(x, w, w, ids)
    with pytest.raises(TypeError):
        b.moe_lora_product(x, w, w, ids, out_dtype=torch.int8)
    with pytest.raises(TypeError):
        b.moe_lora_product([1.0], w, w, ids, out_dtype=torch.float32)
    with pytest.raises(ValueError, match="gradient"):
        b.moe_lora_product(x, w.requires_grad_(), w, ids)


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
    x, la, lb, ids = on(z(4, 64)), on(z(3, 2, 16, 64)), on(z(3, 2, 8, 16)), on(z(4, dtype=torch.int32))
    lora = (x, la, lb, ids, None, off, None, on(z(4, 8)), 0, None)

    def unfit(match, kind=ValueError, **change):
        names = ("x", "la", "lb", "ids", "base", "off", "scaling", "out", "dt", "ws")
        with pytest.raises(kind, match=match):
            calls.lora(*[change.get(n, v) for n, v in zip(names, lora)])
    unfit("lora_a must be", la=on(z(3, 2, 16, 72)))
    unfit("lora_a must be", lb=on(z(3, 2, 8, 24)))
    unfit("lora_a must be", lb=on(z(2, 2, 8, 16)))
    unfit("lora_a must be", lb=on(z(3, 1, 8, 16)))
    unfit("3 or 4 dims", la=on(z(16, 64)))
    unfit("contiguous", la=on(z(3, 2, 64, 16).transpose(2, 3)))
    unfit("BFloat16", kind=TypeError, la=on(z(3, 2, 16, 64, dtype=torch.float16)))
    unfit("Int", kind=TypeError, ids=on(z(4, dtype=torch.int64)))
    unfit("R = 4", ids=on(z(5, dtype=torch.int32)))
    unfit("missing", off=None)
    unfit("L = 3", scaling=on(z(2, dtype=torch.float32)))
    unfit("Float", kind=TypeError, scaling=on(z(3)))
    unfit("base must be \\[4, 8", base=on(z(4, 9)))
    unfit("base must be BFloat16", kind=TypeError, base=on(z(4, 8, dtype=torch.float32)))
    unfit("contiguous", base=on(z(8, 4).T))
    unfit("out must be \\[4, 8", out=on(z(3, 8)))
    unfit("cuda:0", ids=on(z(4, dtype=torch.int32), 1))
    unfit("cuda:0", base=on(z(4, 8), 1))
    assert pretend.calls() == ([], 0)
    calls.lora(*lora[:4], on(z(4, 40)[:, 3:11]), off, None, on(z(4, 48)[:, 8:16]), 0, None)
    assert pretend.weights()[:2] == (40, 48)


@pytest.mark.parametrize("device", [0, 1, 3])
def test_compiled_calls_launch_on_their_tensors_device(fake, on, device):
    calls, pretend = fake
    t = lambda *s, **k: on(z(*s, **k), device)  # noqa: E731
    off, ws = t(3, dtype=torch.int32), t(16, dtype=torch.uint8)
    calls.product(t(4, 64), t(2, 8, 64), off, t(4, 8), 0, ws)
    calls.product_grad(t(4, 8), t(4, 64), t(2, 8, 64), off, True, True, t(4, 64), t(2, 8, 64), 0, ws)
    calls.lora(t(4, 64), t(3, 2, 16, 64), t(3, 2, 8, 16), t(4, dtype=torch.int32), None, off, None, t(4, 8), 0, ws)
    assert pretend.calls() == ([(device, 100 + device)] * 3, 0)


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
