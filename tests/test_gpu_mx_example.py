"""The example block runs, and its 8- and 4-bit rows differ from the float32
block as their element spacing says they may.

An element is off by at most half its spacing: relative 2^-4 for E4M3 (3
fraction bits), 2^-2 for E2M1 (1 fraction bit), uniform within that, so its
rms is at most 2^-4 / sqrt(3) = 0.036 and 2^-2 / sqrt(3) = 0.144 (values below
the smallest normal element, and clamped ones, err by less of the row's rms).  Two
roundings (the rows and the activation) of independent errors through products
that keep relative rms, the activation gathering those of gate and up (at most
2 of the first kind in rms sum): sqrt(1 + 2) times the bound of one."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 64, 300])
@pytest.mark.parametrize("bits,one", [(8, 2.0 ** -4 / 3 ** 0.5), (4, 2.0 ** -2 / 3 ** 0.5)])
def test_example_block(tokens, bits, one):
    spec = importlib.util.spec_from_file_location("mx_moe_block", os.path.join(ROOT, "examples", "mx_moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    err = m.main(["--tokens", str(tokens), "--bits", str(bits)])
    assert 0 < err <= 3 ** 0.5 * one
