"""64-bit references and accuracy criteria of the 4-bit product and of the
cross entropy, on tensors of any device.

An element-wise bound of the worst case grows with the square of a row's
length and hides lost precision there.  These are criteria of the usual error
(Frobenius norms, root mean squares), several times what correct arithmetic
leaves:
  * fp32 results: rounding errors of a sum of n terms accumulate like sqrt(n)
    2^-24 times its partial sums: below 3e-6 of the result for n <= 16384.  Bound:
    1e-5, for Y, dH and dW relative to their norm, for loss and lse relative to
    1 + |lse|.
  * bf16 gradients: one rounding of the result and one of the logits' gradient,
    at most 2^-8 of each term, 1.7e-3 in the root mean square over mantissas,
    independent of each other: 2.4e-3.  Bound: 4e-3.
  * bf16 products: one rounding, 1.7e-3 over many results.  Bound: 2e-3.
dW's rows that are no token's target hold the softmax part of the gradient
alone, which is small beside the target's part elsewhere, and are held to the
same bounds by themselves.
"""
import torch

FP32, BF16_GRADIENT, BF16_PRODUCT = 1e-5, 4e-3, 2e-3


def distance(got, want):
    """Relative Frobenius distance."""
    want = want.double()
    norm = torch.linalg.vector_norm(want)
    return float(torch.linalg.vector_norm(got.double() - want) / norm) if norm > 0 else float(got.double().abs().max())


def cross_entropy(H, W, y, dloss):
    """loss, lse, dH, dW in 64 bits, of finite operands; the vocabulary in pieces of 8192."""
    V = W.shape[0]
    on = (y >= 0) & (y < V)
    H = H.double()
    up = torch.where(on, dloss.double(), torch.zeros_like(dloss, dtype=torch.float64)).unsqueeze(1)
    pieces = range(0, V, 8192)
    z = torch.cat([torch.mm(H, W[v:v + 8192].double().t()) for v in pieces], dim=1)
    lse = torch.logsumexp(z, dim=1)
    rows = on.nonzero().squeeze(1)
    target = torch.zeros_like(lse)
    target[rows] = z[rows, y[rows]]
    loss = torch.where(on, lse - target, torch.zeros_like(lse))
    G = torch.exp(z - lse.unsqueeze(1))
    G[rows, y[rows]] -= 1.0
    G *= up
    dH, dW = torch.zeros_like(H), torch.empty(V, H.shape[1], dtype=torch.float64, device=H.device)
    for v in pieces:
        dH += torch.mm(G[:, v:v + 8192], W[v:v + 8192].double())
        dW[v:v + 8192] = torch.mm(G[:, v:v + 8192].t().contiguous(), H)
    return loss, lse, dH, dW


def check_loss(loss, lse, want_loss, want_lse):
    scale = 1 + want_lse.abs()
    for got, want in ((loss, want_loss), (lse, want_lse)):
        assert float((((got.double() - want) / scale) ** 2).mean().sqrt()) <= FP32


def check_gradients(dH, dW, want_dH, want_dW, y):
    bound = BF16_GRADIENT if dH.dtype is torch.bfloat16 else FP32
    V = dW.shape[0]
    rest = torch.ones(V, dtype=torch.bool, device=dW.device)
    rest[y[(y >= 0) & (y < V)]] = False
    off = {"dH": distance(dH, want_dH), "dW": distance(dW, want_dW),
           "dW of no target": distance(dW[rest], want_dW[rest]) if rest.any() else 0.0}
    assert all(v <= bound for v in off.values()), off


def check_product(Y, want):
    off = distance(Y, want)
    assert off <= (BF16_PRODUCT if Y.dtype is torch.bfloat16 else FP32), off


def head(T, V, d, dtype, seed, device="cpu", spread=2.0):
    """Hidden states, head, targets and upstream gradients.  The head's rows share a component, as trained ones do:
    the two parts of dH, sum_v p_v W_v and W_y, then cancel in it and neither can hide a mistake in the other."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device=device, generator=g)  # noqa: E731
    W = ((rand(V, d) + rand(d)) * (spread / d ** 0.5)).to(dtype)
    H = rand(T, d).to(dtype)
    y = torch.randint(0, V, (T,), device=device, generator=g)
    y[torch.rand(T, device=device, generator=g) < 0.1] = -100
    up = torch.rand(T, device=device, generator=g) + 0.5
    return H, W, y, up
