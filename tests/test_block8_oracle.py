"""The oracle of the 8-bit blocks and the gradients, pinned by hand values,
brute force and differences (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block8


def test_e4m3_table_is_the_formats():
    v = block8.e4m3_table()
    assert v[0x00] == 0 and v[0x01] == 2.0 ** -9 and v[0x07] == 7 * 2.0 ** -9
    assert v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x39] == 1.125 and v[0x7E] == 448.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0xFE] == -448.0 and v[0xB8] == -1.0
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)


def test_e4m3_rounding_ties_and_neighbours():
    v = block8.e4m3_table()[:127]
    mid = (v[1:] + v[:-1]) / 2
    c = block8.e4m3_codes(mid)
    assert (c % 2 == 0).all() and (np.abs(c.astype(int) - np.arange(126) - 0.5) == 0.5).all()
    assert np.array_equal(block8.e4m3_codes(mid * (1 - 1e-12)), np.arange(126))
    assert np.array_equal(block8.e4m3_codes(-mid * (1 + 1e-12)), np.arange(1, 127) | 128)
    assert np.array_equal(block8.e4m3_codes(v), np.arange(127))
    assert block8.e4m3_codes(np.array([np.nan, -0.0])).tolist() == [0x7F, 0x80]


@pytest.mark.parametrize("top,n", [(448.0, 0), (448.25, 1), (1.0, -8), (0.875, -9), (0.8750001, -8), (65504.0, 8),
                                   (57344.0, 7), (2.0 ** -24, -32), (1e-45, -126), (0.0, 0)])
def test_pack8_scale_is_the_smallest_power_that_fits(top, n):
    x = np.zeros((1, 128))
    x[0, 5] = -top
    _, s = block8.pack8(x, 1, "f32")
    assert s[0, 0] == 2.0 ** n
    if n > -126 and top:
        assert top > 448 * 2.0 ** (n - 1)


def test_pack8_caps_in_the_top_binade_and_marks_what_is_not_finite():
    x = np.zeros((1, 256))
    x[0, :4] = [65504.0, -65504.0, 60000.0, 1.0]
    x[0, 128:131] = [np.inf, np.nan, 3.0]
    c, s = block8.pack8(x, 1, "f16")
    v = block8.unpack8(c, s, 1)
    assert v[0, :3].tolist() == [61440.0, -61440.0, 61440.0]
    assert np.isnan(v[0, 128]) and np.isnan(v[0, 129]) and v[0, 130] == 3.0
    c32, s32 = block8.pack8(x, 1, "f32")
    assert block8.unpack8(c32, s32, 1)[0, 0] == 65536.0


@pytest.mark.parametrize("block_rows,rows", [(1, 3), (128, 130)])
def test_pack8_error_is_half_a_step(block_rows, rows):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((rows, 384)) * np.exp(rng.standard_normal((rows, 1)))
    c, s = block8.pack8(x, block_rows, "f32")
    each = np.repeat(np.repeat(s, 128, 1), block_rows, 0)[:rows]
    err = np.abs(block8.unpack8(c, s, block_rows) - x)
    # half of 2^-3 of the value's binade, or half of e4m3's subnormal step
    assert (err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * each)).all()
    assert s.shape == (-(-rows // block_rows), 3)


def test_products_against_torch_on_hand_made_blocks():
    w = np.full((1, 128), 0x38, dtype=np.uint8)          # ones
    x = np.full((2, 128), 0x38, dtype=np.uint8)
    x[1] = 0xB8
    y, d = block8.gemm8(w, np.array([[0.5]]), x, np.array([[2.0], [0.25]]))
    assert y.tolist() == [[128.0], [-16.0]] and d.tolist() == [[128.0], [16.0]]


def test_weight_is_the_oracles_matvec():
    rng = np.random.default_rng(9)
    planes, alpha, _ = oracle.pack(rng.standard_normal((37, 256)), 3, 128)
    x = rng.standard_normal((4, 256))
    y, _ = oracle.matvec(planes, alpha, x)
    assert np.allclose(x @ block8.weight(planes, alpha).T, y, rtol=0, atol=1e-12)


def test_gradients_against_differences():
    """L = sum(C * (X W^T)): dX and dW from the formulas against central
    differences of the fp64 forward (linear in each, so exact but for
    rounding); the planes do not depend on X, and the gradient with respect to
    the reconstructed weight is the one the shared weight receives."""
    rng = np.random.default_rng(10)
    planes, alpha, _ = oracle.pack(rng.standard_normal((5, 128)) * 0.02, 2, 0)
    W = block8.weight(planes, alpha)
    X, C = rng.standard_normal((3, 128)), rng.standard_normal((3, 5))
    loss = lambda X, W: float((C * (X @ W.T)).sum())      # noqa: E731
    dX, _ = block8.dgrad(C, planes, alpha)
    dW, _ = block8.wgrad(C, X)
    for _ in range(20):
        t, j, i = rng.integers(3), rng.integers(128), rng.integers(5)
        E = np.zeros_like(X)
        E[t, j] = 0.5
        assert abs(loss(X + E, W) - loss(X - E, W) - dX[t, j]) < 1e-12
        E = np.zeros_like(W)
        E[i, j] = 0.5
        assert abs(loss(X, W + E) - loss(X, W - E) - dW[i, j]) < 1e-12
