"""Workspaces of the 16-bit operators that share memory with a call's inputs or results are
refused (no GPU needed: addresses are never dereferenced)."""

import ctypes

import pytest
import torch

# (a call that were not refused would use the addresses where there is a GPU)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

vp = ctypes.c_void_p
BF16, F32 = 0, 2
A, W, OFF, Y, OUT, DW, WS = (0x100000000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    from weight_quantized_moe_gb300 import binding, build
    build.build()
    return binding.lib()


def shared(lib, rc):
    """Refused for that; the other calls here end in an earlier or a later refusal."""
    return rc == 1 and b"workspace must not share" in lib.mq_last_error_message()


def around(at, size, need):
    """Addresses of a workspace of `need` bytes that meets [at, at + size) by 16 bytes, or less
    where there is less."""
    return (at, at + (size - 1) // 16 * 16, at - need + 16)


def test_product(lib):
    R, K, N = 1, 4096, 256      # stored [K, N]: summed in splits
    need = lib.moe_grouped_product_workspace(R, K, N, 1)
    assert need > 0

    def call(ws, stride=K):
        return lib.moe_grouped_product(vp(A), stride, BF16, R, K, N, 1, vp(W), N, N * K, 1, vp(OFF), vp(OUT), BF16,
                                       vp(ws), need, None)
    for at, size in ((A, 2 * K), (W, 2 * N * K), (OFF, 8), (OUT, 2 * N)):
        for ws in around(at, size, need):
            assert shared(lib, call(ws)), (hex(at), hex(ws))


def test_workspaces_that_are_not_needed_are_not_looked_at(lib):
    """(Nothing runs: without a GPU the launch fails.)"""
    R, K, N, E = 64, 64, 128, 8
    assert lib.moe_grouped_product_workspace(R, K, N, E) == 0
    for ws in (A + 64, W + 64, OUT + 64):
        rc = lib.moe_grouped_product(vp(A), K, BF16, R, K, N, E, vp(W), K, N * K, 0, vp(OFF), vp(OUT), BF16, vp(ws),
                                     1 << 20, None)
        assert not shared(lib, rc)


def test_gradients(lib):
    R, K, N = 4096, 64, 64
    need = lib.moe_grouped_product_grad_workspace(R, K, N, 1)
    assert need > 0

    def call(ws, da=OUT, dw=DW):
        return lib.moe_grouped_product_grad(vp(Y), N, vp(A), K, BF16, R, K, N, 1, vp(W), K, N * K, 0, vp(OFF), vp(da),
                                            vp(dw), F32, vp(ws), need, None)
    for at, size in ((Y, 2 * R * N), (A, 2 * R * K), (W, 2 * N * K), (OFF, 8), (OUT, 2 * R * K), (DW, 4 * N * K)):
        for ws in around(at, size, need):
            assert shared(lib, call(ws)), (hex(at), hex(ws))
    # a misaligned one is refused before anything is launched
    assert call(WS + 8) == 1 and b"aligned" in lib.mq_last_error_message()


def test_adapters(lib):
    R, K, N, r, L = 2000, 64, 72, 16, 3
    B, IDS, SC = 0x900000000, 0xA00000000, 0xB00000000
    need = lib.moe_lora_product_workspace(R, K, N, r, L, 1)
    assert need > 0

    def call(ws, x=A, xs=K, base=Y, bs=N, out=OUT, os=N):
        return lib.moe_lora_product(vp(x), xs, BF16, R, K, N, r, L, 1, vp(W), vp(B), vp(IDS), vp(OFF), vp(SC), vp(base),
                                    bs, vp(out), os, BF16, vp(ws), need, None)
    for at, size in ((A, 2 * R * K), (W, 2 * L * r * K), (B, 2 * L * r * N), (IDS, 4 * R), (OFF, 8), (SC, 4 * L),
                     (Y, 2 * R * N), (OUT, 2 * R * N)):
        for ws in around(at, size, need):
            assert shared(lib, call(ws)), (hex(at), hex(ws))
    # rows that are far apart: their gaps may hold it, their rows not
    wide = 1 << 20
    assert need < 2 * wide - 256
    assert 2 * wide * R <= 1 << 32
    for k in ("xs", "bs", "os"):
        at = {"xs": A, "bs": Y, "os": OUT}[k]
        for row in (0, 1, R // 2):      # (the last rows reach into other arrays' addresses)
            assert shared(lib, call(at + row * 2 * wide, **{k: wide})), (k, row)
            assert shared(lib, call(at + row * 2 * wide - need + 16, **{k: wide})), (k, row)
