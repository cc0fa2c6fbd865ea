"""Special values in 16-bit activations of the 4-bit product: the form for few
tokens quantises them with conversions of its own; needs an MI355X."""
import numpy as np
import pytest

from oracle import mxfp4 as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOKENS = [1, 2, 4, 5, 33]                                 # the first three quantise X inside the product


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vector_codebook_codec_amd as pkg
    from vector_codebook_codec_amd import _lib

    _lib.load()
    return pkg


def check(q, X, codes, scales, name):
    """Every partial sum rounds to at most 2^-23 of the sum of magnitudes, and there are fewer of them than products."""
    print(f"case activations {name} {tuple(X.shape)} {X.dtype}", flush=True)
    Y = q.qamw_mxfp4_matmul(X, codes, scales)
    torch.cuda.synchronize()
    exact, S = M.matmul(X.double().cpu().numpy(), codes.cpu().numpy(), scales.cpu().numpy())
    got = Y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(exact))
    ok = ~np.isnan(exact)
    assert (np.abs(got - exact)[ok] <= X.shape[1] * 2.0 ** -23 * S[ok]).all()
    return got


def unit_weights(q, d, at, size=1.0):
    """Weights that pick one column each: its product is the activation's value, exactly."""
    W = torch.zeros(len(at), d, device=DEV)
    for n, j in enumerate(at):
        W[n, j] = size
    return q.qamw_mxfp4_quantize(W)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_every_element(q, T, dt):
    """All finite values of a type's low exponents, ties among them, one block of 32 to a scale, read back exactly."""
    d = 1024
    bits = np.arange(T * d, dtype=np.int64) * (29 if dt == "bf16" else 31) % 0x7c00
    bits = (bits | (np.arange(T * d) % 2) << 15).astype(np.uint16).reshape(T, d)
    X = torch.from_numpy(bits.view(np.int16)).view(DT[dt]).to(DEV)
    at = list(range(0, d, 7))
    codes, scales = unit_weights(q, d, at)
    got = check(q, X, codes, scales, "every element")
    want = M.dequantize(*M.quantize(X.double().cpu().numpy()), d)[:, at]
    normal = (np.abs(want) >= 2.0 ** -126) | (want == 0)
    assert np.array_equal(got[normal], want[normal])


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_subnormal_activations(q, T, dt):
    """Blocks of the type's subnormal values; the weights bring the products back into fp32's normal range."""
    d = 96
    rng = np.random.default_rng(T)
    bits = rng.integers(0, 0x80 if dt == "bf16" else 0x400, (T, d)) | rng.integers(0, 2, (T, d)) << 15
    X = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(DT[dt]).to(DEV)
    at = list(range(d))
    codes, scales = unit_weights(q, d, at, 2.0 ** 40)
    got = check(q, X, codes, scales, "subnormal")
    want = M.dequantize(*M.quantize(X.double().cpu().numpy()), d) * 2.0 ** 40
    assert np.array_equal(got, want)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_infinities_and_nan(q, T, dt):
    """A block with an infinity or a NaN makes its token's results NaN, and no other's; a zero weight does not hide it."""
    d, N = 160, 70
    rng = np.random.default_rng(T)
    X = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(DT[dt])
    for t, (j, v) in enumerate(((d - 1, np.inf), (0, -np.inf), (77, np.nan))):
        if t + 1 < T:
            X[t + 1, j] = v
    if T == 1:
        X[0, 33] = np.nan
    W = torch.from_numpy(rng.standard_normal((N, d)).astype(np.float32))
    W[5] = 0.0
    codes, scales = q.qamw_mxfp4_quantize(W.to(DEV))
    got = check(q, X.to(DEV), codes, scales, "infinities and NaN")
    assert np.isnan(got).any(axis=1).tolist() == torch.isfinite(X).all(dim=1).logical_not().tolist()


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_wide_scales(q, T, dt):
    """Blocks of scales over the type's range, zeros and the type's largest value among them."""
    d, N = 320, 50
    rng = np.random.default_rng(T + 9)
    lo, hi = (-60, 60) if dt == "bf16" else (-24, 15)
    block = lambda n: np.repeat(2.0 ** rng.integers(lo, hi, size=(n, d // 32)), 32, axis=1)  # noqa: E731
    a = np.clip(rng.standard_normal((T, d)) * block(T), -6e4, 6e4) if dt == "f16" else rng.standard_normal((T, d)) * block(T)
    X = torch.from_numpy(a.astype(np.float32)).to(DT[dt])
    X[:, 64:96] = 0.0
    X[0, 130] = 65504.0 if dt == "f16" else 2.0 ** 62
    codes, scales = q.qamw_mxfp4_quantize(torch.from_numpy((rng.standard_normal((N, d)) * block(N)).astype(np.float32)).to(DEV))
    check(q, X.to(DEV), codes, scales, "wide scales")
