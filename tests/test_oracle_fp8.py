"""Pins of the 8-bit oracle: the e4m3 format, the block quantiser, and the linear over it."""
import numpy as np
import pytest

import workloads as W
from oracle import fp8
from oracle.gated_linear import gated_linear

torch = pytest.importorskip("torch")


def test_code_values_are_the_format():
    v = fp8.code_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(v.astype(np.float32), t)
    assert np.nanmax(v) == 448.0 and np.nanmin(np.abs(v[v != 0])) == 2.0 ** -9


def test_rounding_matches_the_type_at_every_midpoint():
    v = np.sort(fp8.code_values()[:127])
    mids = (v[1:] + v[:-1]) / 2
    pts = np.concatenate([v, mids, mids * (1 + 1e-6), mids * (1 - 1e-6)])
    pts = np.concatenate([pts, -pts]).astype(np.float32)
    got = fp8.round_e4m3(pts)
    np.testing.assert_array_equal(got, torch.from_numpy(pts).to(torch.float8_e4m3fn).double().numpy())
    assert fp8.round_e4m3(1e9) == 448.0 and fp8.round_e4m3(-500.0) == -448.0


@pytest.mark.parametrize("rows,M,K", [(1, 5, 264), (128, 130, 264), (1, 1, 8)])
def test_quantised_values_are_within_half_a_step(rows, M, K):
    x = W.bf16_to_f64(W.bf16_round(np.random.default_rng(0).standard_normal((M, K))))
    v, s = fp8.quantize(x, rows)
    h = fp8.values(v, s, rows)
    sc = np.repeat(np.repeat(s.astype(np.float64), rows, 0)[:M], 128, 1)[:, :K]
    # half a step: 2^-4 of the value, or half the smallest step; 2^-22 for the float32 scale
    assert np.all(np.abs(h - x) <= 2.0 ** -4 * np.abs(x) + (2.0 ** -10) * sc + 2.0 ** -22 * np.abs(x))
    assert np.abs(v).max() == 448.0
    z, sz = fp8.quantize(np.zeros((2, 128)), 1)
    assert not z.any() and np.all(sz > 0)


def test_linear_of_exact_values_is_the_plain_one_and_the_gradient_its_transpose():
    rng = np.random.default_rng(1)
    M, K, N, r = 3, 256, 128, 8
    x = rng.choice([-2.0, -1.0, 1.0, 2.0], (M, K))           # block maxima are powers of two times 448/448: exact
    x[:, ::128] = 448.0
    Wv = rng.choice(fp8.code_values()[:126], (N, K))
    Ws = np.full((1, 2), 0.5, np.float32)
    A, Bl = rng.standard_normal((r, K)), rng.standard_normal((N, r))
    gate = np.array([0, 1, 1])
    y, bound = fp8.gated_linear_fp8(x, Wv, Ws, A, Bl, gate, 0.5)
    np.testing.assert_allclose(y, gated_linear(x, Wv * 0.5, A, Bl, gate, 0.5), rtol=1e-12)
    assert np.all(bound > 0)
    # <dy, y(x)> is linear in x with coefficient dx (dy exact in e4m3 too)
    dy = rng.choice([-2.0, 1.0, 4.0], (M, N))
    dy[:, ::128] = 448.0
    dx, _ = fp8.gated_input_grad_fp8(dy, Wv, Ws, A, Bl, gate, 0.5)
    e = rng.standard_normal((M, K))
    f = lambda z: float((dy * gated_linear(z, Wv * 0.5, A, Bl, gate, 0.5)).sum())   # noqa: E731
    h = 1e-3
    np.testing.assert_allclose((f(x + h * e) - f(x - h * e)) / (2 * h), (dx * e).sum(), rtol=1e-6)
