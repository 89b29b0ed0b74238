"""The FP64 oracle of the paged-attention operators against closed forms and
differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import paged


def test_plan_of_one_request_by_hand():
    # 5 cached tokens in pages of 4 (pages 7, 2), 6 new ones: positions 5..10
    table, lens, pos, slots, end, err = paged.page_plan(
        [5], [0, 6], 6, [[7, 2, -1, -1]], [3, 9, 1], 4, start=1)
    assert table.tolist() == [[7, 2, 9, -1]] and lens.tolist() == [11] and end == 2 and err is None
    assert pos.tolist() == [5, 6, 7, 8, 9, 10]
    assert slots.tolist() == [9, 10, 11, 36, 37, 38]


def test_plan_refuses_what_does_not_fit():
    free = [10, 11, 12]
    # request 0 wants 2 pages, 1 wants 2 (one is left), 2 wants none, 3 wants 1
    table, lens, _, slots, end, err = paged.page_plan(
        [0, 0, 1, 0], [0, 5, 10, 11, 12], 12, np.full((4, 3), 5), free, 4)
    assert err == "pages" and end == 2 and lens.tolist() == [5, 0, 2, 0]
    assert (slots[5:10] == -1).all() and slots[11] == -1 and slots[10] == 21
    # a row that is too short takes nothing and stops nobody
    _, lens, _, _, end, err = paged.page_plan([0, 0], [0, 9, 10], 10, np.zeros((2, 2)), free, 4)
    assert err == "pages" and lens.tolist() == [0, 1] and end == 1
    assert paged.page_plan([0], [0, 3], 4, [[0]], free, 4)[-1] == "arg"


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    rng = np.random.default_rng(0)
    f = 10.0 ** -rng.random(8)
    a, b = rng.standard_normal((2, 20))
    R = lambda p: paged.rotation(16, 20, p, f, interleaved, 1.0)
    assert np.allclose(R(9) @ R(9).T, np.eye(20))
    assert math.isclose((R(13) @ a) @ (R(9) @ b), (R(4) @ a) @ b)


@pytest.mark.parametrize("norm", [False, True])
def test_gradient_against_differences(norm):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 2, 3, 16))
    w, f, pos = rng.random(16) + 0.5, rng.random(4), [3, 50]
    args = (pos, f)
    dx, dw = paged.norm_rope_grad(x, dy, *args, w, 1e-3, norm, True, 1.3)
    val = lambda x, w: (paged.norm_rope(x, *args, w, 1e-3, norm, True, 1.3) * dy).sum()
    h = 1e-6
    for i in [(0, 0, 0), (1, 2, 7), (0, 1, 15)]:
        d = np.zeros_like(x)
        d[i] = h
        # central difference: error h^2 of the third derivative, here below 1e-9
        assert abs((val(x + d, w) - val(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for c in (0, 9):
            d = np.zeros(16)
            d[c] = h
            assert abs((val(x, w + d) - val(x, w - d)) / (2 * h) - dw[c]) < 1e-7


def test_decode_of_equal_keys_is_the_mean_of_the_values():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((3, 1, 4, 8))
    k = np.ones((3, 1, 4, 8))
    q = rng.standard_normal((2, 2, 8))
    out, lse, _, _ = paged.paged_decode(q, k, v, [[2, 0], [1, -1]], [6, 0], 0.5)
    mean = np.concatenate([v[2, 0], v[0, 0, :2]]).mean(0)
    assert np.allclose(out[0], mean) and np.allclose(lse[0], 0.5 * q[0].sum(-1) + math.log(6))
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
