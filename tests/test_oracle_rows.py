"""Pins of the oracle's norm, rotation and cache rows: library conversions, complex products,
autograd, finite differences and closed forms (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle.rows import rotate


def table(max_pos, rot, base=10000.0):
    ang = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


def test_e4m3_round_is_the_library_conversion():
    rng = np.random.default_rng(0)
    codes = oracle.e4m3_decode(np.arange(256, dtype=np.uint8))
    codes = np.sort(codes[np.isfinite(codes)])
    ties = (codes[1:] + codes[:-1]) / 2
    x = np.concatenate([codes, ties, np.nextafter(ties, 9e9), np.nextafter(ties, -9e9), rng.normal(0, 100, 4000),
                        rng.normal(0, 0.01, 4000)]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(oracle.e4m3_round(x), want)
    assert np.array_equal(oracle.e4m3_round([1e9, -np.inf, 460.0]), [448.0, -448.0, 448.0])
    assert np.isnan(oracle.e4m3_round([np.nan])).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, tab, pos = rng.normal(size=(5, 2, 64)), table(40, 32), np.array([0, 3, 39, 17, 1])
    y = rotate(x, tab, pos, interleaved)
    a, b = (x[..., 0:32:2], x[..., 1:32:2]) if interleaved else (x[..., :16], x[..., 16:32])
    z = (a + 1j * b) * (tab[pos, :16] + 1j * tab[pos, 16:])[:, None]
    ya, yb = (y[..., 0:32:2], y[..., 1:32:2]) if interleaved else (y[..., :16], y[..., 16:32])
    assert np.allclose(ya + 1j * yb, z, atol=1e-14) and np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose(rotate(y, tab, pos, interleaved, back=True), x, atol=1e-14)
    # scores depend on the distance alone
    q, k = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    dot = lambda i, j: float((rotate(q, table(40, 64), np.array([i]), interleaved)
                              * rotate(k, table(40, 64), np.array([j]), interleaved)).sum())
    assert abs(dot(11, 4) - dot(37, 30)) < 1e-12


@pytest.mark.parametrize("interleaved,rot,weighted", [(False, 64, True), (True, 32, True), (False, 16, False)])
def test_norm_rope_gradients(interleaved, rot, weighted):
    rng = np.random.default_rng(2)
    x, dy = rng.normal(size=(4, 3, 64)), rng.normal(size=(4, 3, 64))
    w = 1 + 0.3 * rng.normal(size=64) if weighted else None
    tab, pos = table(9, rot), np.array([5, 0, 8, 2])
    dx, dw = oracle.norm_rope_backward(dy, x, w, tab, pos, 1e-3, True, interleaved)
    f = lambda x_, w_: float((oracle.norm_rope(x_, w_, tab, pos, 1e-3, True, interleaved) * dy).sum())
    for _ in range(3):
        v = rng.normal(size=x.shape)
        h = 1e-6
        assert abs((f(x + h * v, w) - f(x - h * v, w)) / (2 * h) - (dx * v).sum()) < 1e-6
        if weighted:
            v = rng.normal(size=64)
            assert abs((f(x, w + h * v) - f(x, w - h * v)) / (2 * h) - (dw * v).sum()) < 1e-6
    # autograd, and the plain rotation's gradient
    xt = torch.from_numpy(x).requires_grad_()
    n = xt * (xt.square().mean(-1, keepdim=True) + 1e-3).rsqrt()
    g = torch.from_numpy(rotate(dy, tab, pos, interleaved, back=True)) * (1 if w is None else torch.from_numpy(w))
    (n * g).sum().backward()
    assert np.allclose(xt.grad.numpy(), dx, atol=1e-12)
    d0, none = oracle.norm_rope_backward(dy, x, None, tab, pos, 0.0, False, interleaved)
    assert none is None and np.allclose((d0 * x).sum(), (dy * rotate(x, tab, pos, interleaved)).sum())


def test_padding_rows():
    x, dy = np.ones((3, 1, 64)), np.ones((3, 1, 64))
    x[1] = np.nan
    pos = np.array([0, -1, 2])
    y = oracle.norm_rope(x, None, table(4, 64), pos, 1e-6)
    assert np.isnan(y[1]).all() and np.isfinite(y[[0, 2]]).all()
    dx, dw = oracle.norm_rope_backward(dy, x, None, table(4, 64), pos, 1e-6)
    assert (dx[1] == 0).all() and np.isfinite(dx).all() and np.isfinite(dw).all()


def test_rows_and_gates_by_hand():
    cu, lens, bt = [0, 2, 2, 3], [17, 5, 1], [[3, 1], [0, 0], [2, 0]]
    assert oracle.row_places(cu, lens, bt, 16) == [(0, 0, 15, 3, 15), (1, 0, 16, 1, 0), (2, 2, 0, 2, 0)]
    g = np.zeros((4, 1, 16))
    g[3, 0, 14] = -5.0
    out = oracle.cache_gates(np.array([[-1.0], [-2.0], [-4.0]]), g, cu, lens, bt, 16)
    assert out[3, 0, 15] == -6.0 and out[1, 0, 0] == -8.0 and out[2, 0, 0] == -4.0 and np.count_nonzero(out) == 4


def test_quantised_rows():
    scale, v = oracle.quantise_row(np.array([448.0, -224.0, 17.0, 0.0], np.float32))
    assert scale == 1.0 and np.array_equal(v, [448.0, -224.0, 16.0, 0.0])  # 17 is a tie: 16 is even
    scale, v = oracle.quantise_row(np.zeros(4, np.float32))
    assert scale == 0.0 and (v == 0).all()
    scale, v = oracle.quantise_row(np.array([1.0, np.nan], np.float32))
    assert np.isnan(scale) and (v == 0).all()
    scale, v = oracle.quantise_row(np.array([1.0, -np.inf], np.float32))
    assert np.isinf(scale) and v[0] == 0 and np.isnan(v[1])
    codes = torch.tensor([1.5, -3.0]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    cache = np.zeros((1, 1, 16, 2), np.uint8)
    cache[0, 0, 3] = codes
    sc = np.zeros((1, 1, 16), np.float32)
    sc[0, 0, 3] = 0.5
    assert np.array_equal(oracle.cache_gather(cache, sc, [0, 1], [4], [[0]], 16)[0, 0], [0.75, -1.5])
    assert np.array_equal(oracle.cache_gather(cache, np.array([2.0]), [0, 1], [4], [[0]], 16)[0, 0], [3.0, -6.0])
