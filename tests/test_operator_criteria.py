"""The accuracy criteria of operator_criteria.py on the CPU: the operators'
arithmetic, emulated, passes them, and arithmetic with a planted mistake does
not."""
import numpy as np
import pytest

import operator_criteria as K
from oracle import cross_entropy as C
from oracle import mxfp4 as M

torch = pytest.importorskip("torch")


def emulate(H, W, y, up, bf16_logits=False, keep=1.0, bf16_g=False):
    """The operators in fp32, results in H's dtype: logits rounded to bf16 or not, softmax times `keep`, G rounded to
    bf16 relative to the largest upstream gradient or not."""
    V = W.shape[0]
    on = (y >= 0) & (y < V)
    rows = on.nonzero().squeeze(1)
    z = H.float() @ W.float().t()
    if bf16_logits:
        z = z.bfloat16().float()
    m = z.amax(dim=1)
    rest = torch.exp(z - m[:, None]).sum(dim=1).log()
    lse = m + rest
    target = torch.zeros_like(m)
    target[rows] = z[rows, y[rows]]
    loss = torch.where(on, (m - target) + rest, torch.zeros_like(m))
    G = torch.exp(z - lse[:, None]) * keep
    G[rows, y[rows]] -= 1.0
    unit = up[on].max()
    G *= torch.where(on, up / unit, torch.zeros_like(up))[:, None]
    if bf16_g:
        G = G.bfloat16().float()
    return loss, lse, (G @ W.float() * unit).to(H.dtype), (G.t() @ H.float() * unit).to(H.dtype)


@pytest.mark.parametrize("T,V,d", [(5, 1003, 4096), (64, 4090, 1024)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_cross_entropy_criteria(T, V, d, dt):
    H, W, y, up = K.head(T, V, d, dt, T + V)
    want = K.cross_entropy(H, W, y, up)
    loss, lse, dH, dW = emulate(H, W, y, up, bf16_g=dt is torch.bfloat16)
    K.check_loss(loss, lse, *want[:2])
    K.check_gradients(dH, dW, *want[2:], y)
    loss, lse, dH, dW = emulate(H, W, y, up, bf16_logits=True)
    with pytest.raises(AssertionError):
        K.check_loss(loss, lse, *want[:2])
    with pytest.raises(AssertionError):
        K.check_gradients(want[2].to(dt), dW, *want[2:], y)
    for keep in (0.9, 0.98):
        _, _, dH, dW = emulate(H, W, y, up, keep=keep)
        with pytest.raises(AssertionError):                          # in dH alone and in dW alone
            K.check_gradients(dH, want[3].to(dt), *want[2:], y)
        with pytest.raises(AssertionError):
            K.check_gradients(want[2].to(dt), dW, *want[2:], y)


def test_reference_is_the_oracles():
    H, W, y, up = K.head(9, 77, 24, torch.float32, 1)
    got = K.cross_entropy(H, W, y, up)
    loss, lse = C.forward(H.numpy(), W.numpy(), y.numpy())
    dH, dW = C.backward(H.numpy(), W.numpy(), y.numpy(), up.numpy())
    for a, b in zip(got, (loss, lse, dH, dW)):
        assert np.allclose(a.numpy(), b, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("d", [8200, 11008])
def test_product_criteria(d):
    rng = np.random.default_rng(d)
    X, W = rng.standard_normal((40, d)), rng.standard_normal((50, d))
    codes, scales = M.quantize(W)
    want = torch.from_numpy(M.matmul(X, codes, scales)[0])
    xq = torch.from_numpy(M.dequantize(*M.quantize(X), d)).float()
    wq = torch.from_numpy(M.dequantize(codes, scales, d)).float()
    K.check_product(xq @ wq.t(), want)
    K.check_product((xq @ wq.t()).bfloat16(), want)
    with pytest.raises(AssertionError):                              # a bf16 result in fp32
        K.check_product((xq @ wq.t()).bfloat16().float(), want)
    shares = sum((xq[:, k:k + 512] @ wq[:, k:k + 512].t()).bfloat16().float() for k in range(0, d, 512))
    with pytest.raises(AssertionError):                              # bf16 sums of shares of the contraction
        K.check_product(shares, want)
