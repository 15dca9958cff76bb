"""The fp64 definitions of the training operators against closed forms,
independent formats and differences (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import training_oracle as ref


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_code_values_are_the_formats(fmt):
    got = ref.code_values(fmt)
    bits = torch.arange(256, dtype=torch.uint8)
    want = (bits.view(torch.float8_e4m3fn) if fmt == "e4m3" else bits.view(torch.int8)).double().numpy()
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_checkpoint_is_the_nearest_value_of_the_smallest_scale(fmt):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((6, 70)) * np.exp2(rng.integers(-30, 30, (6, 1)))).astype(np.float32).astype(np.float64)
    x[2, :32] = 0.0
    got, scales = ref.checkpoint(x, fmt)
    grid = np.unique(ref.code_values(fmt)[np.isfinite(ref.code_values(fmt))])
    grid = grid[np.abs(grid) <= ref.LARGEST[fmt]]
    for r in range(6):
        for b in range(3):
            v, e = x[r, 32 * b:32 * b + 32], int(scales[r, b]) - 127
            assert np.abs(v).max() <= math.ldexp(ref.LARGEST[fmt], e)
            assert e == -111 or np.abs(v).max() > math.ldexp(ref.LARGEST[fmt], e - 1)
            near = np.abs(v[:, None] - np.ldexp(grid, e)[None]).min(axis=1)
            np.testing.assert_array_equal(np.abs(got[r, 32 * b:32 * b + 32] - v), near)
    # half steps go to the even code
    row = np.zeros((1, 32))
    row[0, :5] = [ref.LARGEST[fmt], 2.5, 3.5, -2.5, 0.5]
    got, _ = ref.checkpoint(row, fmt)
    if fmt == "int8":
        assert got[0, :5].tolist() == [127.0, 2.0, 4.0, -2.0, 0.0]
    else:
        row[0, 1:5] = [1.0625, 1.1875, -17.0, 0.0009765625]
        assert ref.checkpoint(row, fmt)[0][0, :5].tolist() == [448.0, 1.0, 1.25, -16.0, 0.0]


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(4)
    g, u, d = 3 * rng.standard_normal((3, 40))
    grad_gate, grad_up, h = ref.swiglu_backward(d, g, u)
    np.testing.assert_allclose(h, ref.swiglu(g, u), rtol=1e-14)
    step = 1e-5     # central differences: error of order step^2 plus 2^-53 / step
    np.testing.assert_allclose(grad_gate, d * (ref.swiglu(g + step, u) - ref.swiglu(g - step, u)) / (2 * step), rtol=0, atol=1e-8)
    np.testing.assert_allclose(grad_up, d * (ref.swiglu(g, u + step) - ref.swiglu(g, u - step)) / (2 * step), rtol=0, atol=1e-8)


def test_wgrad_is_the_gradient_of_the_product():
    """sum(grad_y * (x W^T)) is linear in W: its slope is dW."""
    rng = np.random.default_rng(5)
    x, dy, w = rng.standard_normal((9, 5)), rng.standard_normal((9, 4)), rng.standard_normal((4, 5))
    dw = ref.wgrad(dy, x)
    assert math.isclose((dw * w).sum(), (dy * (x @ w.T)).sum(), rel_tol=1e-12)
    np.testing.assert_array_equal(ref.wgrad(dy, x, transposed=True), dw.T)
    rows = np.array([3, 0, 8, -1, 3, 2, 9, 1, 5])
    parts = ref.wgrad(dy, x, offsets=[2, 5, 5, 8], rows=rows)
    assert parts.shape == (3, 4, 5)
    np.testing.assert_allclose(parts[0], np.outer(dy[2], x[8]) + np.outer(dy[4], x[3]), rtol=1e-14)
    assert not parts[1].any()
    np.testing.assert_allclose(parts[2], np.outer(dy[5], x[2]) + np.outer(dy[7], x[1]), rtol=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(6)
    logits, ids = rng.standard_normal((4, 7)), np.array([[2, 0, 5], [6, 1, -1], [-1, -1, -1], [3, 4, 0]])
    dw = rng.standard_normal((4, 3))
    got = ref.route_backward(dw, logits, ids, score, renormalize, 1.7)
    step = 1e-5
    for t in range(4):
        for e in range(7):
            up, down = logits[t].copy(), logits[t].copy()
            up[e] += step
            down[e] -= step
            diff = (ref.route_weights(up, ids[t], score, renormalize, 1.7) - ref.route_weights(down, ids[t], score, renormalize, 1.7)) / (2 * step)
            assert abs(got[t, e] - (dw[t] * diff).sum()) < 1e-8


def test_route_definition_on_small_rows():
    r = ref.route([[0.0, 2.0, 2.0, -math.inf], [-math.inf] * 4, [1.0, math.nan, 0.0, 0.0], [5.0, 1.0, 1.0, 1.0]], 3)
    assert r["experts"].tolist() == [[1, 2, 0], [-1] * 3, [-1] * 3, [0, 1, 2]]
    assert np.isnan(r["weights"][2]).all() and not r["weights"][1].any()
    assert r["counts"].tolist() == [2, 2, 2, 0] and r["offsets"].tolist() == [0, 2, 4, 6, 6]
    assert r["order"].tolist() == [2, 9, 0, 10, 1, 11, -1, -1, -1, -1, -1, -1]
    assert r["rows"].tolist() == [0, 3, 0, 3, 0, 3] + [-1] * 6
    # a bias moves the choice and not the weight
    r = ref.route([[0.0, 0.0, 0.0]], 1, bias=[0.0, 0.0, 0.5], renormalize=False)
    assert r["experts"].tolist() == [[2]] and math.isclose(r["weights"][0, 0], 1 / 3)
    # the second run of two has the better pair, the first the best single choice
    logits = [[3.0, -3.0, 1.0, 1.0]]
    assert ref.route(logits, 1, score="sigmoid", groups=2, top_groups=1)["experts"].tolist() == [[2]]
    assert ref.route(logits, 1, score="sigmoid", groups=2, top_groups=1, group_top=1)["experts"].tolist() == [[0]]
    assert ref.route(logits, 2, token_mask=[0])["experts"].tolist() == [[-1, -1]]


def test_balance_moves_toward_the_mean():
    got = ref.balance([0.0, 0.0, 0.0, 0.0], [5, 1, 3, 3], 0.25)
    assert got.tolist() == [-0.25, 0.25, 0.0, 0.0]
    assert ref.balance([1.0], [7], 0.25).tolist() == [1.0]
