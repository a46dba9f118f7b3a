"""Pins of the fp64 definitions of RMS norm and of the block formats."""
import numpy as np
import pytest

from oracle import head as O


def test_rms_norm_by_hand():
    y, rstd = O.rms_norm([[3.0, -4.0], [0.0, 0.0]], [1.0, 0.5], 1.0, 1e-30)
    r = 1.0 / np.sqrt(12.5)
    assert np.allclose(rstd[0], r) and np.allclose(y[0], [6.0 * r, -6.0 * r])
    assert np.array_equal(y[1], [0.0, 0.0])


@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_rms_norm_gradients_against_differences(offset):
    g = np.random.default_rng(1)
    s, w, dy, ds = g.normal(size=(3, 7)), g.normal(size=7), g.normal(size=(3, 7)), g.normal(size=(3, 7))
    eps = 0.03

    def loss(s, w):
        return (O.rms_norm(s, w, offset, eps)[0] * dy).sum() + (ds * s).sum()

    dx, dw = O.rms_norm_grads(dy, s, w, offset, O.rms_norm(s, w, offset, eps)[1], ds)
    h = 1e-6
    for got, at, which in ((dx, s, 0), (dw, w, 1)):
        for i in np.ndindex(at.shape):
            d = np.zeros(at.shape)
            d[i] = h
            a = (s + d, w) if which == 0 else (s, w + d)
            b = (s - d, w) if which == 0 else (s, w - d)
            assert abs((loss(*a) - loss(*b)) / (2 * h) - got[i]) < 1e-7


def test_formats_match_torch():
    torch = pytest.importorskip("torch")
    codes = torch.arange(128, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), O.e4m3_values(), equal_nan=True)
    y = np.random.default_rng(2).normal(size=(50, 64)) * 10.0 ** np.random.default_rng(3).uniform(-9, 9, size=(50, 1))
    y = y.astype(np.float32)
    code, e = O.mx_quantize(y, O.e4m3_values())
    scaled = torch.from_numpy(y / np.repeat(2.0 ** e.astype(np.float64), 32, 1).astype(np.float32))
    assert np.array_equal(scaled.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), code)


def test_quantize_by_hand():
    code, e = O.mx_quantize([[6.0, 5.0, -2.5, 0.25, 0.75, -0.2] + [0.0] * 27], O.E2M1)
    assert e.tolist() == [[0, -127]]
    assert code[0, :6].tolist() == [7, 6, 8 | 4, 0, 2, 0]   # ties to the even code
    code, e = O.mx_quantize([[6.001], [3.0], [448.0]], O.E2M1)
    assert e.tolist() == [[1], [-1], [7]] and code.tolist() == [[5], [7], [6]]   # 448 = 2^7 3.5: tie to 4
    _, e = O.mx_quantize([[448.0], [448.5], [0.0], [1e-45]], O.e4m3_values())
    assert e.tolist() == [[0], [1], [-127], [-127]]
