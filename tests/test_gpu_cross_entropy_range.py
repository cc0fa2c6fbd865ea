"""Gradients of large logits and of confident tokens; needs an MI355X.

The logits here are exact in fp32 (small integers times powers of two, few
columns), so that only the softmax's own arithmetic is left (U = 2^-24):
  * the sum of exponentials: about 30 additions in a row, each term's exp off
    by 2 U and its argument x = lse - z by 3 U x (x times its share of the sum
    adds up to at most 5): 64 U together, which is also its logarithm's error;
  * lse is rounded to fp32, |lse| U, and (top - z_y) + rest by 4 U of it;
  * p = exp(z - lse): those two, 8 U for its own roundings, 3 U x for its
    argument; probabilities below 2^-126 may be 0;
  * sums of n products: n U of the sum of their magnitudes."""
import numpy as np
import pytest

from oracle import cross_entropy as C

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vector_codebook_codec_amd as pkg
    from vector_codebook_codec_amd import _lib

    _lib.load()
    return pkg


def check(q, H, W, y, g):
    Ht, Wt, yt, gt = (torch.from_numpy(a).to(DEV) for a in (H.astype(np.float32), W.astype(np.float32), y, g.astype(np.float32)))
    loss, lse = q.qamw_cross_entropy(Ht, Wt, yt)
    dH, dW = q.qamw_cross_entropy_grad(Ht, Wt, yt, lse, gt)
    torch.cuda.synchronize()
    z = H @ W.T
    assert np.array_equal(z.astype(np.float32).astype(np.float64), z)
    want, want_lse = C.forward(H, W, y)
    on = C.counted(y, W.shape[0])
    tol = (np.abs(want_lse) + 4 + 64) * U
    assert (np.abs(lse.cpu().double().numpy() - want_lse) <= tol).all()
    assert (np.abs(loss.cpu().double().numpy() - want) <= np.abs(want) * 4 * U + 64 * U).all()
    G = C.logit_grad(H, W, y, g)
    x = np.minimum(want_lse[:, None] - z, 90.0)
    p = np.where(on[:, None], np.exp(-x), 0.0) * np.abs(g)[:, None]
    dG = p * (np.abs(want_lse)[:, None] + 64 + 8 + 3 * x) * U + np.abs(G) * 4 * U + 2.0 ** -124
    for got, exact, off in ((dH, G @ W, dG @ np.abs(W) + W.shape[0] * U * (np.abs(G) @ np.abs(W))),
                            (dW, G.T @ H, dG.T @ np.abs(H) + H.shape[0] * U * (np.abs(G).T @ np.abs(H)))):
        assert (np.abs(got.cpu().double().numpy() - exact) <= off).all()
    return loss.cpu().double().numpy(), want


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("size", [1.0, 64.0, 1024.0, 8192.0])
def test_large_logits(q, T, size):
    """Logits of up to 8192 and of either sign, far past exp's range, a few units apart."""
    print(f"case large logits T={T} size {size}", flush=True)
    rng = np.random.default_rng(int(size) + T)
    V, d = 120, 8
    W = rng.integers(-8, 9, (V, d)) / 64.0
    W[:, 0] = 1.0                                        # H's first column shifts all logits of a token
    H = rng.integers(-32, 33, (T, d)) / 16.0
    H[:, 0] = size * np.where(np.arange(T) % 2, -1.0, 1.0)
    y = rng.integers(0, V, T)
    y[T - 1] = -100
    check(q, H, W, y, rng.standard_normal(T).astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("T", [4, 60])
def test_confident_tokens(q, T):
    """Targets with all but 1e-2 to 1e-6 of the mass at log sums of up to 100: the loss keeps its digits (six roundings
    of a sum just above 1, one of its logarithm), where lse alone would be off by up to 64 U; G_y keeps its stated
    distance."""
    print(f"case confident tokens T={T}", flush=True)
    V, d = 16, 8
    W = np.zeros((V, d))
    W[:, 0], W[:, 1] = 1.0, -(np.arange(V) % 4 + 1.0)
    W[5, 1] = 0.0
    H = np.zeros((T, d))
    H[:, 0] = np.arange(T) % 8 * 16.0 - 12.0             # the target's logit: -12 to 100
    H[:, 1] = 16.0 - np.arange(T) % 10                   # its distance from the others
    y = np.full(T, 5)
    loss, want = check(q, H, W, y, np.ones(T))
    assert want.min() < 1e-6 and (np.abs(loss - want) <= 8 * U).all()
