"""What autograd has to know of calls that write to, or read, its tensors: on the CPU with the
compiled calls on stand-in devices, on the GPU with recorded calls."""

import ctypes

import pytest
import torch

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def grouped(tmp_path_factory):
    from grouped_fake_device import compile_fake
    return compile_fake(str(tmp_path_factory.mktemp("grouped")))


@pytest.fixture(scope="module")
def mx(tmp_path_factory):
    from mx_fake_device import compile_fake
    return compile_fake(str(tmp_path_factory.mktemp("mx")))


class Maker:
    """Zeros on a pretended device (and their host memory, kept)."""

    def __init__(self, fake):
        self.fake, self.keep = fake, []

    def __call__(self, *shape, dtype=BF16):
        self.keep.append(torch.zeros(*shape, dtype=dtype))
        return self.fake.on_device(self.keep[-1], 0)


def versions_rise(call, given):
    before = [t._version for t in given]
    call()
    assert all(t._version > b for t, b in zip(given, before))


def test_given_results_of_the_16_bit_calls_change_version(grouped):
    calls, t = grouped[0], Maker(grouped[1])
    a, w, off, out = t(4, 64), t(2, 8, 64), t(3, dtype=I32), t(4, 8)
    versions_rise(lambda: calls.product(a, w, off, out, 0, None), [out])
    da, dw = t(4, 64), t(2, 8, 64)
    versions_rise(lambda: calls.product_grad(out, a, w, off, True, True, da, dw, 0, None), [da, dw])
    h = t(4, 8)
    ids, la, lb = t(4, dtype=I32), t(3, 2, 16, 64), t(3, 2, 8, 16)
    versions_rise(lambda: calls.lora(a, la, lb, ids, h, off, None, h, 0, None), [h])
    assert [x._version for x in (a, w, off, ids, la, lb)] == [0] * 6
    with pytest.raises(ValueError):    # a refused call writes nothing
        calls.product(a, w, None, out, 0, None)
    assert out._version == 1


def test_given_results_of_the_microscaled_calls_change_version(mx):
    calls, t = mx[0], Maker(mx[1])
    x, q, s = t(4, 64), t(4, 64, dtype=U8), t(4, 2, dtype=U8)
    versions_rise(lambda: calls.quantize(x, 8, q, s), [q, s])
    out = t(4, 64)
    versions_rise(lambda: calls.dequantize(q, s, 8, 0, out), [out])
    y, ro = t(4, 64), t(4, 64)
    versions_rise(lambda: calls.rmsnorm(x, t(64), 1e-6, x, 8, True, ro, y, q, s), [q, s, y, ro])
    p, w, ws = t(4, 8), t(8, 32, dtype=U8), t(8, 2, dtype=U8)
    versions_rise(lambda: calls.product(q, s, w, ws, None, 8, p, 0, None), [p])
    assert x._version == 0 and w._version == 0


def test_inference_tensors_are_written_as_before(grouped):
    calls, t = grouped[0], Maker(grouped[1])
    a, w = t(4, 64), t(1, 8, 64)
    with torch.inference_mode():
        out = t(4, 8).view(4, 8)
    assert out.is_inference()
    calls.product(a, w, None, out, 0, None)


def test_given_results_of_the_quantised_calls_change_version(monkeypatch):
    """(The library is a stand-in that says everything went well, and tensors of the host pass
    for the device's.)"""
    from weight_quantized_moe_gb300 import binding as b

    class Library:
        def __getattr__(self, name):
            return lambda *args: 0
    monkeypatch.setattr(b, "lib", lambda: Library())
    monkeypatch.setattr(b, "_need", lambda *args: None)
    monkeypatch.setattr(b, "_stream", lambda stream=None: ctypes.c_void_p(0))
    T, H, I, E, k = 4, 64, 32, 2, 1
    x, logits = torch.zeros(T, H, dtype=BF16), torch.zeros(T, E)
    w13, w2 = torch.zeros(E, 2 * I, H, dtype=torch.int8), torch.zeros(E, H, I, dtype=torch.int8)
    s13, s2 = torch.zeros(E, 2 * I), torch.zeros(E, H)
    tw, ids, out = torch.zeros(T, k), torch.zeros(T, k, dtype=I32), torch.zeros(T, H, dtype=BF16)
    versions_rise(lambda: b.moe_topk_route(logits, k, True, topk_w=tw, topk_ids=ids), [tw, ids])
    args = (w13, w2, s13, s2, tw, ids)
    versions_rise(lambda: b.moe_quant_forward(x, *args, out=out), [out])
    versions_rise(lambda: b.moe_quant_forward_noalloc(x, *args, out=out), [out])
    versions_rise(lambda: b.moe_quant_forward_logits(x, logits, w13, w2, s13, s2, k, out=out), [out])
    assert x._version == 0
    versions_rise(lambda: b.moe_quant_forward(x, *args, inplace=True), [x])
    versions_rise(lambda: b.moe_quant_forward_logits(x, logits, w13, w2, s13, s2, k, inplace=True), [x])
    q, s = torch.zeros(E, H, I, dtype=torch.int8), torch.zeros(E, H)
    versions_rise(lambda: b.moe_quantize_int8_per_channel(torch.zeros(E, H, I, dtype=BF16), q=q, scale=s), [q, s])


def test_tangents_are_refused(grouped):
    """A result without a tangent would be a derivative of zero."""
    import torch.autograd.forward_ad as fwd
    calls, t = grouped[0], Maker(grouped[1])
    a, w, off, out = t(4, 64), t(2, 8, 64), t(3, dtype=I32), t(4, 8)
    da, dw = t(4, 64), t(2, 8, 64)
    product = (a, w, off, out, 0, None)
    grad = (t(4, 8), a, w, off, True, True, da, dw, 0, None)
    lora = (a, t(3, 2, 16, 64), t(3, 2, 8, 16), t(4, dtype=I32), t(4, 8), off, t(3, dtype=F32), out, 0, None)
    for call, args, floats in ((calls.product, product, (0, 1, 3)), (calls.product_grad, grad, (0, 1, 2, 6, 7)),
                               (calls.lora, lora, (0, 1, 2, 4, 6, 7))):
        call(*args)
        for i in floats:
            with fwd.dual_level():
                dual = list(args)
                dual[i] = fwd.make_dual(args[i], t(*args[i].shape, dtype=args[i].dtype))
                assert not dual[i].requires_grad
                with pytest.raises(ValueError, match="tangent"):
                    call(*dual)
        call(*args)


def test_calls_without_a_gradient_refuse_tensors_that_require_one(grouped, monkeypatch):
    from weight_quantized_moe_gb300 import binding as b
    calls, t = grouped[0], Maker(grouped[1])
    monkeypatch.setattr(b, "_grouped", calls)
    dy, a, w, off = t(4, 8), t(4, 64), t(2, 8, 64), t(3, dtype=I32)
    da, dw, out = t(4, 64), t(2, 8, 64), t(4, 8)
    given = dict(dy=dy, a=a, w=w, expert_offsets=off, da=da, dw=dw)
    b.moe_grouped_product_grad(**given)
    for name in ("dy", "a", "w", "da", "dw"):
        leaf = given[name].detach().requires_grad_()
        with pytest.raises(ValueError, match="no_grad"):
            b.moe_grouped_product_grad(**{**given, name: leaf})
        with torch.no_grad():
            b.moe_grouped_product_grad(**{**given, name: leaf})
    b.moe_grouped_product(a, w, off, out=out)
    leaf = out.detach().requires_grad_()
    with pytest.raises(ValueError, match="out"):
        b.moe_grouped_product(a, w, off, out=leaf)
    with torch.no_grad():
        b.moe_grouped_product(a, w, off, out=leaf)


@pytest.mark.gpu
def test_a_saved_input_that_was_written_is_refused():
    """h is saved for a backward pass; adapters added to it in place change its version."""
    import weight_quantized_moe_gb300 as mq
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    x, w1, w2 = r(8, 64), r(64, 64), r(72, 64).requires_grad_()
    a, b, ids = r(2, 8, 64), r(2, 64, 8), torch.zeros(8, dtype=I32, device="cuda")

    def recorded():
        h = mq.moe_grouped_product(x, w1)
        return h, mq.moe_grouped_product(h, w2)
    h, y = recorded()
    with torch.no_grad():
        mq.moe_lora_product(x, a, b, ids, base=h, out=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    h, y = recorded()
    mq.moe_grouped_product(x, w1, out=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    wide = torch.zeros(8, 192, dtype=BF16, device="cuda")      # (a slice is written: the whole counts)
    versions_rise(lambda: mq.moe_lora_product(x, a, b, ids, out=wide[:, 64:128]), [wide])
    h, y = recorded()
    mq.moe_lora_product(x, a, b, ids, base=h)          # not in place
    y.sum().backward()
    assert w2.grad is not None
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0


@pytest.mark.gpu
def test_tangents_are_refused_where_the_call_is_recorded():
    import torch.autograd.forward_ad as fwd

    import weight_quantized_moe_gb300 as mq
    x, w = torch.zeros(8, 64, dtype=BF16, device="cuda"), torch.zeros(72, 64, dtype=BF16, device="cuda")
    for grad in (False, True):
        w = w.detach().requires_grad_(grad)
        with fwd.dual_level(), pytest.raises((ValueError, RuntimeError, NotImplementedError)):
            mq.moe_grouped_product(fwd.make_dual(x, torch.ones_like(x)), w)
    mq.moe_grouped_product(x, w).sum().backward()
