"""GPU parity of the 4-bit product with low-rank adapters against the oracle
(oracle/mxfp4.py); needs an MI355X.

Criteria, element by element:
  * the shared product as in test_gpu_mxfp4.py: d 2^-23 S, S the sum of its
    products' magnitudes;
  * the adapters: sums of d and of r fp32 products, rounded to at most 2^-23 of
    S2 = |f| sum_k |B| sum_j |A| |X| each time, and the factor: (d + r + 2)
    2^-23 S2; U as two bf16 numbers is off by 2^-16 of each entry: 2^-16 sum_k
    |U| |B| for bf16;
  * the sum of both: 2^-23 (S + S2), and the result's half step, 2^-8 for bf16;
over all elements, where there are 256 or more, in the root mean square: 2e-3 for bf16 results, 2e-5 for fp32
ones with bf16 adapters (2^-16 / sqrt(3) of U at most, 9e-6), 1e-5 for fp32.
A token's result does not depend on other tokens' adapters: rows without one
equal qamw_mxfp4_matmul's bit for bit.
"""
import sys

import numpy as np
import pytest

from oracle import mxfp4 as M

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


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def host(t):
    return t.detach().cpu().double().numpy()


def make(q, T, N, d, r, n, dt, seed):
    rng = np.random.default_rng(seed)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    X = new(T, d).to(DT[dt]).to(DEV)
    codes, scales = q.qamw_mxfp4_quantize((new(N, d) * 0.02).to(DEV))
    A = (new(n, r, d) * d ** -0.5).to(DT[dt]).to(DEV)
    B = (new(n, N, r) * 0.1).to(DT[dt]).to(DEV)
    f = torch.from_numpy((rng.random(n) + 0.5).astype(np.float32)).to(DEV)
    return rng, X, codes, scales, A, B, f


def check(got, X, codes, scales, A, B, index, f, dt, out):
    d, r = X.shape[1], A.shape[1]
    want, S, S2, inner = M.adapter_matmul(host(X), codes.cpu().numpy(), scales.cpu().numpy(), host(A), host(B), index, host(f))
    got = host(got)
    bound = d * 2.0 ** -23 * S + (d + r + 2) * 2.0 ** -23 * S2 + 2.0 ** -23 * (S + S2)
    if dt == "bf16":
        bound += 2.0 ** -16 * inner
    if out == "bf16":
        bound += 2.0 ** -8 * np.abs(want)
    off = np.abs(got - want)
    assert (off <= bound).all(), (off / np.maximum(bound, 1e-300)).max()
    most = 2e-3 if out == "bf16" else 2e-5 if dt == "bf16" else 1e-5
    if got.size >= 256:                            # a mean of one or a few half steps is no mean
        assert np.linalg.norm(got - want) <= most * np.linalg.norm(want)


# T, N, d, r, adapters, how the tokens choose
CASES = [
    (1, 1, 1, 1, 1, "each"), (1, 300, 64, 8, 3, "each"), (2, 33, 100, 3, 2, "each"), (4, 513, 96, 16, 1, "each"),
    (5, 70, 1003, 5, 9, "each"), (16, 520, 256, 17, 16, "each"), (20, 100, 512, 32, 7, "runs"), (33, 8300, 64, 16, 5, "each"),
    (70, 200, 320, 33, 70, "each"), (64, 64, 64, 64, 2, "none"), (100, 1000, 96, 7, 100, "each"), (129, 257, 513, 24, 4, "runs"),
    (300, 900, 128, 64, 3, "runs"), (257, 300, 96, 100, 40, "each"), (65, 130, 2000, 128, 2, "runs"), (30, 40, 64, 260, 4, "each"),
]


def choose(rng, T, n, how):
    if how == "none":
        return np.full(T, -1, dtype=np.int32)
    if how == "each":
        index = rng.integers(0, n, T)
    else:
        index = np.sort(rng.integers(0, n, T))
    index = index.astype(np.int32)
    if T > 2:
        index[rng.random(T) < 0.2] = -1
        index[T // 2] = n                          # not an adapter
    return index


@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,N,d,r,n,how", CASES)
def test_adapters(q, T, N, d, r, n, how, dt, out):
    say(f"case adapters T={T} N={N} d={d} r={r} n={n} {how} {dt} -> {out}")
    rng, X, codes, scales, A, B, f = make(q, T, N, d, r, n, dt, T * 7 + d)
    index = choose(rng, T, n, how)
    got = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, torch.from_numpy(index).to(DEV), f, out_dtype=DT[out])
    torch.cuda.synchronize()
    check(got, X, codes, scales, A, B, index, f, dt, out)
    base = q.qamw_mxfp4_matmul(X, codes, scales, out_dtype=DT[out])
    bare = torch.from_numpy((index < 0) | (index >= n))
    assert torch.equal(got.cpu()[bare], base.cpu()[bare])
