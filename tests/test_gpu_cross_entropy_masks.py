"""Tokens that are not counted, against heads with infinite and NaN weights;
needs an MI355X."""
import numpy as np
import pytest

from oracle import cross_entropy as C

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vector_codebook_codec_amd as pkg
    from vector_codebook_codec_amd import _lib

    _lib.load()
    return pkg


@pytest.mark.parametrize("T,V,d,dt", [
    (1, 700, 64, "bf16"), (3, 700, 64, "f32"), (4, 700, 64, "bf16"), (16, 1100, 4096, "bf16"),     # few tokens
    (140, 300, 256, "bf16"), (140, 300, 256, "f32"),                                               # dH written by its product
    (40, 5003, 64, "bf16"), (40, 5003, 64, "f32"),                                                 # dH summed over shares
    (700, 300, 1024, "bf16"), (2300, 130, 1024, "f32")])                                           # larger tiles
@pytest.mark.parametrize("all_masked", [False, True])
def test_rows_of_zeros_under_any_head(q, T, V, d, dt, all_masked):
    """dH of a token that is not counted is 0 by definition, not 0 times the head; its loss is 0, and it adds nothing to dW."""
    print(f"case infinite head T={T} V={V} d={d} {dt}, all masked: {all_masked}", flush=True)
    rng = np.random.default_rng(T + V)
    W = torch.from_numpy((rng.standard_normal((V, d)) * 0.1).astype(np.float32)).to(DT[dt])
    W[7], W[20, 3], W[V - 1, d - 1] = float("inf"), float("nan"), float("-inf")
    H = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(DT[dt])
    y = rng.integers(0, V, T)
    y[rng.random(T) < 0.3] = -100
    y[0] = V
    if all_masked:
        y[:] = -1
    on = C.counted(y, V)
    H, W, y = H.to(DEV), W.to(DEV), torch.from_numpy(y).to(DEV)
    g = torch.ones(T, device=DEV)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    alone, _ = q.qamw_cross_entropy_grad(H, W, y, lse, g, need_dW=False)
    torch.cuda.synchronize()
    off = torch.from_numpy(~on).to(DEV)
    assert (loss[off] == 0).all() and (dH[off] == 0).all() and (alone[off] == 0).all()
    if all_masked:
        assert (dW == 0).all()
    else:                                                # the head's NaN reaches every token that counts
        assert torch.isnan(loss[~off]).all() and torch.isnan(dH[~off]).all()
