"""Accuracy of the cross entropy, its gradient and the 4-bit product over long
rows, large tiles, shares of the contraction and several pieces of the
vocabulary, by the norm criteria of operator_criteria.py; needs an MI355X.

The references are 64-bit products on the same GPU (plain two-dimensional
ones)."""
import numpy as np
import pytest

import operator_criteria as K
from oracle import mxfp4 as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vector_codebook_codec_amd as pkg
    from vector_codebook_codec_amd import _lib

    _lib.load()
    return pkg


def check_training(q, T, V, d, dt, repeats=1):
    H, W, y, up = K.head(T, V, d, DT[dt], T + V, DEV)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, up)
    for _ in range(repeats):
        again, same = q.qamw_cross_entropy(H, W, y)
        dH2, dW2 = q.qamw_cross_entropy_grad(H, W, y, lse, up)
        assert torch.equal(again, loss) and torch.equal(same, lse) and torch.equal(dH2, dH) and torch.equal(dW2, dW)
    only_dH, _ = q.qamw_cross_entropy_grad(H, W, y, lse, up, need_dW=False)
    _, only_dW = q.qamw_cross_entropy_grad(H, W, y, lse, up, need_dH=False)
    torch.cuda.synchronize()
    assert torch.equal(only_dH, dH) and torch.equal(only_dW, dW)
    want = K.cross_entropy(H, W, y, up)
    K.check_loss(loss, lse, *want[:2])
    K.check_gradients(dH, dW, *want[2:], y)


@pytest.mark.parametrize("T,V,d,dt", [
    (1, 5003, 512, "bf16"), (4, 2050, 8192, "f32"), (5, 1003, 4096, "bf16"), (16, 1100, 4096, "bf16"),
    (17, 3001, 4096, "f32"), (64, 4090, 4096, "bf16"), (64, 4090, 4096, "f32"), (300, 5003, 512, "f32"),
    (4001, 4090, 64, "bf16"), (4090, 300, 4096, "bf16"), (2050, 200, 2048, "f32"), (1030, 1500, 8192, "bf16"),
    (130, 32000, 1024, "bf16")])
def test_training_accuracy(q, T, V, d, dt):
    print(f"case training accuracy T={T} V={V} d={d} {dt}", flush=True)
    check_training(q, T, V, d, dt)


@pytest.mark.parametrize("T,V,d,dt", [
    (2048, 40001, 4096, "bf16"),                         # large tiles
    (40, 70001, 4096, "bf16"),                           # small tiles, shares of the contraction
    (2100, 12300, 8192, "f32")])
def test_several_pieces(q, T, V, d, dt):
    """Heads whose gradient walks the vocabulary in pieces of matrix products, the last one shorter, with targets in
    all of them.  In one piece, G, its transpose and the transposed head alone would take this much memory:"""
    es = DT[dt].itemsize
    assert q.qamw_cross_entropy_grad_workspace_bytes(T, V, d, DT[dt]) < (2 * T + d) * V * es
    print(f"case several pieces T={T} V={V} d={d} {dt}", flush=True)
    check_training(q, T, V, d, dt, repeats=3)


@pytest.mark.parametrize("T", [3, 16])
def test_several_pieces_few_tokens(q, T):
    """The same in the form for few tokens, whose workspace grows with the pieces: less for this head than for a
    smaller one, which is thus one piece where this is several."""
    V, d = 70001, 4096
    size = q.qamw_cross_entropy_grad_workspace_bytes
    assert size(T, V, d, torch.bfloat16) < size(T, 60000, d, torch.bfloat16)
    print(f"case several pieces T={T} V={V} d={d}", flush=True)
    check_training(q, T, V, d, "bf16", repeats=3)


@pytest.mark.parametrize("T,N,d,xdt,ydt", [
    (1, 4097, 11008, "bf16", "f32"), (4, 515, 8200, "f16", "bf16"), (13, 4096, 11008, "f32", "f32"),
    (32, 4096, 8200, "bf16", "f32"), (130, 300, 8192, "bf16", "f32"), (1000, 900, 8200, "bf16", "f32"),
    (1000, 5120, 13824, "bf16", "f32"), (1000, 5120, 13824, "bf16", "bf16"), (4100, 4099, 1056, "bf16", "f32")])
def test_product_accuracy(q, T, N, d, xdt, ydt):
    print(f"case product accuracy T={T} N={N} d={d} {xdt} -> {ydt}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(T + N)
    X = torch.randn(T, d, device=DEV, generator=g).to(DT[xdt])
    codes, scales = q.qamw_mxfp4_quantize(torch.randn(N, d, device=DEV, generator=g) * 0.02)
    Y = q.qamw_mxfp4_matmul(X, codes, scales, out_dtype=DT[ydt])
    # X's codes are checked byte for byte against the oracle on some rows, the values of both operands multiplied in 64 bits
    xc, xs, xv = q.qamw_mxfp4_quantize(X, values_dtype=torch.float32)
    wv = q.qamw_mxfp4_dequantize(codes, scales, d)
    some = sorted({0, T // 2, T - 1})
    want_c, want_s = M.quantize(X[some].double().cpu().numpy())
    assert np.array_equal(xc[some].cpu().numpy(), want_c) and np.array_equal(xs[some].cpu().numpy(), want_s)
    assert np.array_equal(xv[some].double().cpu().numpy(), M.dequantize(want_c, want_s, d))
    K.check_product(Y, torch.mm(xv.double(), wv.double().t()))
