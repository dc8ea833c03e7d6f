"""On which device and stream the microscaled calls launch (no GPU needed: the
compiled calls run on stand-ins for the devices and the library)."""

import pytest
import torch

from mx_fake_device import compile_fake
from weight_quantized_moe_gb300 import binding


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return compile_fake(str(tmp_path_factory.mktemp("mx_fake")))


def arguments(on):
    """Each compiled call's arguments, with every output and workspace given."""
    u8, f16, f32, i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
    z = lambda *shape, dtype=u8: on(torch.zeros(*shape, dtype=dtype))  # noqa: E731
    a, s = z(4, 128), z(4, 4)
    return {
        "quantize": (z(4, 128, dtype=f16), 8, a, s),
        "dequantize": (a, s, 8, 0, z(4, 128, dtype=f16)),
        "rmsnorm": (z(4, 128, dtype=f16), z(128, dtype=f16), 1e-6, None, 8, False, None, None, a, s),
        "product": (a, s, z(2, 64, 64), z(2, 64, 4), z(3, dtype=i32), 8, z(4, 64, dtype=f16), 0, z(16)),
        "forward": (a, s, z(2, 256, 64), z(2, 256, 4), z(2, 128, 64), z(2, 128, 4), z(4, 1, dtype=f32),
                    z(4, 1, dtype=i32), 8, z(4, 128, dtype=f16), 0, z(16)),
    }


NAMES = ("quantize", "dequantize", "rmsnorm", "product", "forward")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("device", [0, 1, 3])
def test_calls_launch_on_their_tensors_device(fake, name, device):
    """Device 0 is current: the call makes its tensors' device current and takes
    that device's stream, and leaves device 0 current."""
    calls, pretend = fake
    pretend.calls()
    keep = []   # host memory behind the tensors

    def on(t):
        keep.append(t)
        return pretend.on_device(t, device)
    getattr(calls, name)(*arguments(on)[name])
    assert pretend.calls() == ([(device, 100 + device)], 0)


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_call_leaves_the_device_as_it_was(fake, name):
    calls, pretend = fake
    pretend.calls()
    keep = []

    def on(t):
        keep.append(t)
        return pretend.on_device(t, 2)
    args = list(arguments(on)[name])
    args[-1 if name in ("dequantize", "product", "forward") else -2] = pretend.on_device(keep[0], 1)
    with pytest.raises((TypeError, ValueError)):
        getattr(calls, name)(*args)
    assert pretend.calls() == ([], 0)


class Stream:
    """Enough of a stream to be told apart by its device."""

    def __init__(self, device):
        self.device = torch.device("cuda", device)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(fake, monkeypatch, name):
    """It would not be used: the call runs on its tensors' device."""
    calls, pretend = fake
    pretend.calls()
    entered = []

    class Current:
        def __init__(self, stream):
            entered.append(stream.device.index)

        def __enter__(self):
            pass

        def __exit__(self, *exc):
            pass

    monkeypatch.setattr(torch.cuda, "stream", Current)
    monkeypatch.setattr(binding, "_mx", calls)
    keep = []

    def on(t):
        keep.append(t)
        return pretend.on_device(t, 1)
    args = arguments(on)[name]
    call = {
        "quantize": lambda st: binding.moe_quantize_mx(*args, stream=st),
        "dequantize": lambda st: binding.moe_dequantize_mx(*args[:3], out=args[4], stream=st),
        "rmsnorm": lambda st: binding.moe_rmsnorm_mx(*args, stream=st),
        "product": lambda st: binding.moe_mx_product(*args[:7], workspace=args[8], stream=st),
        "forward": lambda st: binding.moe_mx_forward(*args[:10], workspace=args[11], stream=st),
    }[name]
    with pytest.raises(ValueError, match="stream must be on cuda:1"):
        call(Stream(0))
    assert pretend.calls() == ([], 0) and not entered
    call(Stream(1))
    assert pretend.calls() == ([(1, 101)], 0) and entered == [1]


@pytest.mark.parametrize("name", ("dequantize", "product", "forward"))
def test_codes_and_scales_of_their_own_types_are_taken(fake, name):
    """E4M3 codes as float8_e4m3fn and scales as float8_e8m0fnu: the bytes are the same."""
    calls, pretend = fake
    pretend.calls()
    keep = []

    def on(t):
        if t.dtype == torch.uint8 and t.shape in ((4, 4), (2, 64, 4), (2, 256, 4), (2, 128, 4)):
            t = t.view(torch.float8_e8m0fnu)
        elif t.dtype == torch.uint8 and t.shape == (4, 128):
            t = t.view(torch.float8_e4m3fn)
        keep.append(t)
        return pretend.on_device(t, 0)
    args = arguments(on)[name]
    assert args[1].dtype == torch.float8_e8m0fnu
    getattr(calls, name)(*args)
    assert pretend.calls() == ([(0, 100)], 0)
    # not the other way round
    swapped = (args[1].view(torch.uint8), args[0].view(torch.uint8).view(torch.float8_e8m0fnu), *args[2:])
    with pytest.raises((TypeError, ValueError)):
        getattr(calls, name)(*swapped)
