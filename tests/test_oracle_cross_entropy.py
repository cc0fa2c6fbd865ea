"""Pins of the cross-entropy oracle (no GPU): a closed form, the gradient
against central differences, tokens that are not counted."""
import numpy as np

from oracle import cross_entropy as C


def test_uniform_logits():
    H, W = np.zeros((3, 4)), np.ones((7, 4))
    loss, lse = C.forward(H, W, [0, 6, -100])
    assert np.allclose(lse, np.log(7)) and np.allclose(loss, [np.log(7), np.log(7), 0.0])
    G = C.logit_grad(H, W, [0, 6, -100], [1.0, 2.0, 5.0])
    assert np.isclose(G[0, 0], 1 / 7 - 1) and np.isclose(G[1, 0], 2 / 7) and not G[2].any()


def test_large_logits_do_not_overflow():
    loss, lse = C.forward(np.array([[1e4], [-1e4]]), np.array([[1.0], [0.5]]), [0, 0])
    assert np.allclose(lse, [1e4, -5e3]) and np.allclose(loss, [0.0, 5e3])


def test_gradient_against_differences():
    rng = np.random.default_rng(0)
    T, V, d = 5, 11, 6
    H, W = rng.standard_normal((T, d)), rng.standard_normal((V, d))
    y, g = np.array([3, 10, -1, 11, 0]), rng.standard_normal(T)
    dH, dW = C.backward(H, W, y, g)
    total = lambda a, b: float(C.forward(a, b, y)[0] @ np.where(C.counted(y, V), g, 0.0))  # noqa: E731
    h = 1e-5
    for A, dA, f in ((H, dH, lambda a: total(a, W)), (W, dW, lambda a: total(H, a))):
        for i in np.ndindex(A.shape):
            up, dn = A.copy(), A.copy()
            up[i] += h
            dn[i] -= h
            # central differences: truncation h^2 f'''/6 ~ 1e-9, rounding 1e-16 * |f| / h ~ 1e-9
            assert abs((f(up) - f(dn)) / (2 * h) - dA[i]) < 1e-7


def test_uncounted_hidden_states_are_not_read():
    rng = np.random.default_rng(1)
    H, W = rng.standard_normal((3, 4)), rng.standard_normal((5, 4))
    H[1] = np.nan
    with np.errstate(invalid="ignore"):
        dH, dW = C.backward(H, W, [1, -100, 2], [1.0, 1.0, 1.0])
    assert np.isfinite(dH).all() and np.isfinite(dW).all() and not dH[1].any()
