"""Pins of the fp64 oracle of the operators around attention: hand-worked page
bookkeeping, the rotation's definition, gradients against differences."""
import numpy as np
import pytest

import oracle


def test_extend_pages_by_hand():
    table = np.array([[7, 0, 0], [0, 0, 0], [5, 6, 0]])
    out, faults = oracle.extend_pages(table, [15, 0, 32], [2, 0, 1], [1, 2, 3, 4], 3, 5, 8)
    assert not faults
    assert out["table"].tolist() == [[7, 3, 0], [0, 0, 0], [5, 6, 2]]
    assert out["lens"].tolist() == [17, 0, 33] and out["cu"].tolist() == [0, 2, 2, 3]
    assert out["positions"].tolist() == [15, 16, 32, 0, 0]
    assert out["slots"].tolist() == [7 * 16 + 15, 3 * 16, 2 * 16, -1, -1]
    assert out["left"] == 1


def test_extend_pages_stops_at_the_first_that_does_not_fit():
    out, faults = oracle.extend_pages(np.zeros((3, 4), int), [0, 0, 0], [16, 17, 1], [0, 1, 2], 2,
                                      100, 3)
    assert faults == {"pages"}
    assert out["lens"].tolist() == [16, 0, 0] and out["left"] == 1


def test_rotation_turns_a_pair_by_the_angle():
    a = np.array([[0.3, 1.1], [0.0, -2.0]])
    table = np.concatenate([np.cos(a), np.sin(a)], 1)
    x = np.array([[[1.0, 2.0, 3.0, 4.0]], [[1.0, 2.0, 3.0, 4.0]]])
    R = oracle.rotation(table, np.array([[0, 1]]), None, 4, False)
    y = oracle.norm_rope(x, None, R, 0.0)
    z = (x[:, 0, :2] + 1j * x[:, 0, 2:]) * np.exp(1j * a)       # halves as complex numbers
    assert np.allclose(y[:, 0], np.concatenate([z.real, z.imag], 1))
    R = oracle.rotation(table, np.array([[0, 1]]), None, 4, True)
    y = oracle.norm_rope(x, None, R, 0.0)
    z = (x[:, 0, 0::2] + 1j * x[:, 0, 1::2]) * np.exp(1j * a)   # neighbours
    assert np.allclose(y[:, 0, 0::2], z.real) and np.allclose(y[:, 0, 1::2], z.imag)


@pytest.mark.parametrize("weighted", [True, False])
def test_norm_rope_gradient_matches_differences(weighted):
    rng = np.random.default_rng(3)
    T, H, D, rot = 2, 3, 16, 8
    ang = rng.normal(size=(5, rot // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    R = oracle.rotation(table, rng.integers(0, 5, (2, T)), [0, 1, 1, 0], D, True)
    x, dy = rng.normal(size=(T, H, D)), rng.normal(size=(T, H, D))
    w = rng.normal(size=D) if weighted else None
    dx, dw = oracle.norm_rope_backward(x, w, R, dy, 1e-3)
    h = 1e-6

    def f(x, w):
        return (oracle.norm_rope(x, w, R, 1e-3) * dy).sum()

    for at in [(0, 0, 0), (1, 2, 7), (1, 0, 15)]:
        step = np.zeros_like(x)
        step[at] = h
        assert abs((f(x + step, w) - f(x - step, w)) / (2 * h) - dx[at]) < 1e-7
    if weighted:
        for d in (0, 5, 15):
            step = np.zeros(D)
            step[d] = h
            assert abs((f(x, w + step) - f(x, w - step)) / (2 * h) - dw[d]) < 1e-7
    else:
        assert dw is None
