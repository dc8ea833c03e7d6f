"""Pins of the microscaled oracle: tables, rounding, scales, round trips,
brute force on tiny inputs."""

import numpy as np
import pytest

from oracle import mx_oracle as mx


def test_element_tables():
    assert mx.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert mx.E4M3[0] == 0 and mx.E4M3[1] == 2.0 ** -9 and mx.E4M3[8] == 2.0 ** -6
    assert mx.E4M3[-1] == 448 and np.all(np.diff(mx.E4M3) > 0)
    torch = pytest.importorskip("torch")
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(codes.float().numpy().astype(np.float64), mx.E4M3)


@pytest.mark.parametrize("v,want", [(0.25, 0), (0.2500001, 0.5), (0.75, 1), (1.25, 1), (1.75, 2),
                                    (2.5, 2), (3.5, 4), (5, 4), (5.0001, 6), (7.9, 6), (100, 6)])
def test_e2m1_rounding(v, want):
    for s in (1, -1):
        c = int(mx.round_to_element(np.array([s * v]), 4)[0])
        assert mx.E2M1[c & 7] == want and c >> 3 == (s < 0)


def test_e4m3_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    v = np.random.default_rng(0).standard_normal(20000) * np.exp2(np.random.default_rng(1).integers(-12, 9, 20000))
    v = np.float32(np.clip(v, -448, 448))
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(mx.round_to_element(v.astype(np.float64), 8), want)


@pytest.mark.parametrize("bits", [4, 8])
def test_scale_rule(bits):
    emax = 2 if bits == 4 else 8
    for a, e in [(1.0, 0), (1.999, 0), (2.0, 1), (0.5, -1), (2.0 ** -140, -127 + emax), (0.0, -127 + emax)]:
        assert int(mx.scale_codes(a, bits)) == max(e - emax, -127) + 127, a
    assert int(mx.scale_codes(np.inf, bits)) == 255 and int(mx.scale_codes(np.nan, bits)) == 255


@pytest.mark.parametrize("bits", [4, 8])
def test_round_trip_of_representable_values(bits):
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 8 if bits == 4 else 127, (5, 64)).astype(np.uint8)
    codes[:, ::BLOCK_FIRST] = 7 if bits == 4 else 126   # every block holds its largest element
    scale = rng.integers(1, 240, (5, 2)).astype(np.uint8)
    v = mx.mx_dequantize(mx.pack(codes, bits), scale, bits)
    q, s = mx.mx_quantize(v, bits)
    assert np.array_equal(s, scale) and np.array_equal(q, mx.pack(codes, bits))


BLOCK_FIRST = mx.BLOCK


@pytest.mark.parametrize("bits", [4, 8])
def test_quantise_is_the_nearest_element(bits):
    v = np.random.default_rng(3).standard_normal((4, 96))
    q, s = mx.mx_quantize(v, bits)
    got = mx.mx_dequantize(q, s, bits)
    table = mx.element_values(bits)
    grid = np.concatenate([-table[::-1], table])
    step = np.repeat(np.exp2(s.astype(float) - 127), 32, axis=-1)
    best = np.min(np.abs(v[..., None] / step[..., None] - grid), axis=-1) * step
    inside = np.abs(v) <= table[-1] * step
    assert np.allclose(np.abs(got - v)[inside], best[inside], rtol=1e-12, atol=0)
    assert np.all(np.abs(got[~inside]) == (table[-1] * step)[~inside])


def test_nonfinite_blocks():
    v = np.ones((1, 64))
    v[0, 3] = np.inf
    q, s = mx.mx_quantize(v, 8)
    assert s.tolist() == [[255, 119]] and not q[0, :32].any()
    assert np.isnan(mx.mx_dequantize(q, s, 8)[0, :32]).all()


def test_product_and_forward_brute_force():
    rng = np.random.default_rng(4)
    a, w = rng.standard_normal((5, 8)), rng.standard_normal((3, 4, 8))
    out, mag = mx.mx_product(a, w, [0, 2, 2, 5])
    for r, e in enumerate([0, 0, 2, 2, 2]):
        for n in range(4):
            assert np.isclose(out[r, n], sum(a[r, k] * w[e, n, k] for k in range(8)))
            assert mag[r, n] >= abs(out[r, n])
    a, w13, w2 = rng.standard_normal((3, 32)), rng.standard_normal((2, 64, 32)), rng.standard_normal((2, 32, 32))
    ids, tw = np.array([[0, 1], [1, 0], [1, -1]]), rng.random((3, 2))
    got = mx.mx_forward(a, w13, w2, tw, ids, 8)
    for t in range(3):
        want = np.zeros(32)
        for j in range(2):
            e = ids[t, j]
            if e < 0:
                continue
            h = w13[e] @ a[t]
            act = h[:32] / (1 + np.exp(-h[:32])) * h[32:]
            want += tw[t, j] * (w2[e] @ mx.mx_dequantize(*mx.mx_quantize(act[None], 8), 8)[0])
        assert np.allclose(got[t], want)


def test_rmsnorm_brute_force():
    x = np.array([[3.0, 4.0]])
    h, y = mx.rmsnorm(x, np.array([[1.0, -1.0]]), np.array([2.0, 1.0]), 0.5)
    assert h.tolist() == [[4.0, 3.0]]
    assert np.allclose(y, [[4 / np.sqrt(13) * 2, 3 / np.sqrt(13)]])
