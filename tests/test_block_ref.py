"""The 64-bit forms that the GPU tests of the microscaled 4-bit operators and of
layer norm compare with: checked on hand-made values and against differences."""
import numpy as np
import pytest

from tests import _block_ref as ref


def test_codes_round_to_nearest_even():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, 5.1, 0.26, 2.4, 3.6, -6.0, 0.0]])
    code, byte = ref.codes_and_bytes(x, "nv")
    assert byte[0, 0] == 0x38  # e4m3 of 1
    assert list(ref.code_values(code[0])) == [0, 1, 1, 2, 2, 4, 4, 6, 0, -1, 6, 0.5, 2, 4, -6, 0]


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (6.0, 0x38), (6 * 448.0, 0x7E), (1e9, 0x7E), (6 * 2.0 ** -9, 1),
                                       (6 * 2.0 ** -11, 0), (np.inf, 0x7F), (np.nan, 0x7F)])
def test_nv_scales(amax, byte):
    x = np.full((1, 16), amax, dtype=np.float32)
    assert ref.codes_and_bytes(x, "nv")[1][0, 0] == byte


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (1.0, 125), (7.9, 127), (8.0, 128), (2.0 ** 127, 252),
                                       (2.0 ** -126, 0), (2.0 ** -124, 1), (1e-44, 0), (np.inf, 255), (np.nan, 255)])
def test_mx_scales(amax, byte):
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, 3] = amax
    assert ref.codes_and_bytes(x, "mx")[1][0, 0] == byte


def test_packed_layout_by_hand():
    code = np.zeros((130, 64), dtype=np.uint8)
    code[129, 63] = 9
    byte = np.zeros((130, 4), dtype=np.uint8)
    byte[33, 2] = 77
    byte[129, 3] = 5
    q, s = ref.pack(code, byte)
    assert q.shape == (130, 32) and q[129, 31] == 0x90
    assert s.shape == (2, 1, 512) and s[0, 0, 16 * 1 + 4 * 1 + 2] == 77 and s[1, 0, 16 * 1 + 3] == 5


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantized_values_are_near(fmt):
    x = np.random.default_rng(3).standard_normal((40, 96)).astype(np.float32)
    ts = 0.01 if fmt == "nv" else 1.0
    v = ref.quantized(x, fmt, ts) * ts
    # half a step of the top binade is 1 of 6 (nv); the power-of-two scale may cut values at 6 of 8
    amax = np.abs(x.reshape(40, -1, ref.BLOCK[fmt])).max(axis=2).repeat(ref.BLOCK[fmt], axis=1)
    assert np.all(np.abs(v - x) <= amax * (0.26 if fmt == "mx" else 0.19))


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(4)
    X, g, dY = rng.standard_normal((3, 9)), rng.standard_normal(9), rng.standard_normal((3, 9))
    dx, dg, db = ref.layer_norm_backward(dY, X, g, 1e-5)
    h = 1e-6

    def loss(X, g, b):
        return float((ref.layer_norm(X, g, b, 1e-5)[0] * dY).sum())

    z = np.zeros(9)
    for i in range(3):
        for j in range(9):
            e = np.zeros_like(X)
            e[i, j] = h
            assert abs((loss(X + e, g, z) - loss(X - e, g, z)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(9):
        e = np.zeros(9)
        e[j] = h
        assert abs((loss(X, g + e, z) - loss(X, g - e, z)) / (2 * h) - dg[j]) < 1e-7
        assert abs((loss(X, g, e) - loss(X, g, -e)) / (2 * h) - db[j]) < 1e-7
