"""The fp64 oracle of the adapters and the vocabulary losses, against central
differences of its own forward values and against facts of the formulas.

A central difference with step e is off by e^2/6 times the third derivative
plus 2^-52 |f| / e; with e = 1e-5 and values of order 10 both stay below 1e-9."""
import numpy as np
import pytest

import oracle

TOL = 1e-7


def _layer(rng, m=7, rows=9, cols=6, n=3, r=2):
    return (rng.standard_normal((m, cols)), rng.standard_normal((rows, cols)),
            rng.standard_normal((n, r, cols)), rng.standard_normal((n, rows, r)),
            rng.standard_normal(n), np.array([0, 2, -1, 2, 5, 0, 2]))


def _difference(f, a, at, e=1e-5):
    b = a.copy()
    b[at] += e
    up = f(b)
    b[at] -= 2 * e
    return (up - f(b)) / (2 * e)


def test_adapter_gradients_are_the_differences():
    rng = np.random.default_rng(1)
    x, W, A, B, s, idx = _layer(rng)
    dy = rng.standard_normal((len(x), len(W)))
    dx, dA, dB = oracle.adapters_backward(dy, x, W, A, B, s, idx)
    f = lambda x, A, B: float((dy * oracle.adapters_forward(x, W, A, B, s, idx)).sum())  # noqa: E731
    for at in np.ndindex(x.shape):
        assert abs(dx[at] - _difference(lambda v: f(v, A, B), x, at)) < TOL
    for at in np.ndindex(A.shape):
        assert abs(dA[at] - _difference(lambda v: f(x, v, B), A, at)) < TOL
    for at in np.ndindex(B.shape):
        assert abs(dB[at] - _difference(lambda v: f(x, A, v), B, at)) < TOL
    assert not dA[1].any() and not dB[1].any()  # no token takes adapter 1


def test_tokens_outside_the_adapters_take_the_layer_alone():
    rng = np.random.default_rng(2)
    x, W, A, B, s, idx = _layer(rng)
    y = oracle.adapters_forward(x, W, A, B, s, idx)
    for t in (2, 4):
        assert np.array_equal(y[t], (x @ W.T)[t])


@pytest.mark.parametrize("kind", ["labels", "teacher"])
def test_head_gradients_are_the_differences(kind):
    rng = np.random.default_rng(3)
    h, W = rng.standard_normal((5, 6)), rng.standard_normal((11, 6))
    g = rng.standard_normal(5)
    if kind == "labels":
        idx, logits, T = np.array([3, -100, 10, 11, 0]), None, 1.0
    else:
        idx = np.array([[3, 3, 1], [-1, 4, 5], [0, 1, 2], [9, -1, 10], [-1, -1, 11]])
        logits, T = rng.standard_normal((5, 3)) * 3, 1.7
        logits[2, 1] = -np.inf
    dh = oracle.head_backward(h, W, idx, g, logits, T)
    f = lambda v: float((g * oracle.head_loss(v, W, idx, logits, T)[0]).sum())  # noqa: E731
    for at in np.ndindex(h.shape):
        assert abs(dh[at] - _difference(f, h, at)) < TOL
    loss = oracle.head_loss(h, W, idx, logits, T)[0]
    out = [1, 3] if kind == "labels" else [4]
    assert not loss[out].any() and not dh[out].any()
    # a Kullback-Leibler divergence from part of a vocabulary is positive
    assert (np.delete(loss, out) > 0).all()


def test_distilling_one_entry_is_the_cross_entropy():
    rng = np.random.default_rng(4)
    h, W = rng.standard_normal((6, 5)), rng.standard_normal((8, 5))
    y = rng.integers(0, 8, 6)
    a = oracle.head_loss(h, W, y)[0]
    b = oracle.head_loss(h, W, y[:, None], np.full((6, 1), 3.0))[0]
    assert np.allclose(a, b, rtol=0, atol=1e-14)


def test_a_student_that_is_its_teacher_has_no_loss():
    """Entries that hold the whole vocabulary with the student's own logits."""
    rng = np.random.default_rng(5)
    h, W = rng.standard_normal((4, 5)), rng.standard_normal((7, 5))
    idx = np.tile(np.arange(7), (4, 1))
    loss = oracle.head_loss(h, W, idx, h @ W.T, 2.5)[0]
    dh = oracle.head_backward(h, W, idx, np.ones(4), h @ W.T, 2.5)
    assert np.abs(loss).max() < 1e-14 and np.abs(dh).max() < 1e-14
