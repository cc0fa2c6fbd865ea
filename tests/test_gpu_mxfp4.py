"""GPU parity of the microscaled 4-bit operators against the oracle
(oracle/mxfp4.py); needs an MI355X.

Criteria:
  * quantise: codes and scales equal byte for byte; values equal bit for bit
    (rounded to nearest even where the value type is narrower);
  * dequantise: the same values;
  * product: every partial sum of the fp32 accumulation rounds to at most
    2^-23 of the sum S of the products' magnitudes, and there are fewer of
    them than products: |Y - exact| <= d 2^-23 S, plus 2^-8 |exact| for a bf16
    result.
"""
import sys

import numpy as np
import pytest

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


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def weights(N, d, dt, seed, spread=0.5):
    rng = np.random.default_rng(seed)
    a = rng.standard_normal((N, d)) * np.exp(spread * rng.standard_normal((N, d)))
    return torch.from_numpy(a.astype(np.float32)).to(DT[dt])


def host(t):
    return t.detach().cpu().double().numpy()


def check_quantise(q, W, vdt):
    codes, scales, values = q.qamw_mxfp4_quantize(W, values_dtype=DT[vdt])
    c2, s2 = q.qamw_mxfp4_quantize(W)
    back = q.qamw_mxfp4_dequantize(codes, scales, W.shape[1], out_dtype=DT[vdt])
    torch.cuda.synchronize()
    want_c, want_s = M.quantize(host(W))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    want = torch.from_numpy(M.dequantize(want_c, want_s, W.shape[1])).to(torch.float32).to(DT[vdt])
    for got in (values, back):
        assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=12345.0), torch.nan_to_num(want.float(), nan=12345.0))


@pytest.mark.parametrize("dt,vdt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("N,d", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 511), (257, 1003), (64, 4096), (7, 8192 + 8)])
def test_quantise(q, N, d, dt, vdt):
    say(f"case quantise {N} x {d} {dt} -> {vdt}")
    check_quantise(q, weights(N, d, dt, N * 31 + d).to(DEV), vdt)


def test_quantise_special_values(q):
    """Ties, saturation, signed zeros, blocks of zeros, subnormals, the type's largest value, infinities and NaN."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.0, 7.9, 4.0, 0.0, -0.0, 0.249, 0.251, 1.0])
    rows = []
    for e in (-149, -130, -126, -125, -20, 0, 30, 120):
        with np.errstate(over="ignore"):
            rows.append(np.concatenate([ties, -ties[::-1], np.ldexp(1.0, 0) * np.ones(8)]) * 2.0 ** e)
    W = np.zeros((len(rows) + 5, 80), dtype=np.float32)
    for i, r in enumerate(rows):
        W[i, :40] = r
    k = len(rows)
    W[k, 3] = np.inf
    W[k + 1, 40] = -np.inf
    W[k + 2, 79] = np.nan
    W[k + 3, :] = np.finfo(np.float32).max
    W[k + 4, 1] = np.finfo(np.float32).tiny / 4
    say("case quantise special values")
    check_quantise(q, torch.from_numpy(W).to(DEV), "f32")
    check_quantise(q, torch.from_numpy(W).to(DEV).to(torch.bfloat16), "bf16")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_quantise_strided_rows(q, dt):
    """Rows that start off 16-byte boundaries, inside a wider matrix; outputs inside wider ones, whose rest stays."""
    say(f"case quantise strided {dt}")
    N, d = 19, 133
    big = weights(N, d + 12, dt, 5).to(DEV)
    W = big[:, 3:3 + d]
    out = torch.full((N, d + 7), -77.0, dtype=DT[dt], device=DEV)
    codes, scales, _ = q.qamw_mxfp4_quantize(W, values=out[:, 2:2 + d])
    out2 = torch.full_like(out, -77.0)
    q.qamw_mxfp4_dequantize(codes, scales, d, out=out2[:, 2:2 + d])
    torch.cuda.synchronize()
    want_c, want_s = M.quantize(host(W))
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales.cpu().numpy(), want_s)
    want = torch.from_numpy(M.dequantize(want_c, want_s, d)).to(torch.float32).to(DT[dt])
    for o in (out, out2):
        assert torch.equal(o[:, 2:2 + d].cpu(), want)
        assert (o[:, :2] == -77).all() and (o[:, 2 + d:] == -77).all()


def test_quantise_past_32_bit_offsets(q):
    say("case quantise 540000 x 4096 bf16")
    N, d = 540000, 4096                                   # 2.2e9 elements
    W = torch.zeros(N, d, dtype=torch.bfloat16, device=DEV)
    tail = weights(5, d, "bf16", 9).to(DEV)
    W[-5:] = tail
    codes, scales, values = q.qamw_mxfp4_quantize(W, values_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    want_c, want_s = M.quantize(host(tail))
    assert np.array_equal(codes[-5:].cpu().numpy(), want_c) and np.array_equal(scales[-5:].cpu().numpy(), want_s)
    assert np.array_equal(host(values[-5:]), M.dequantize(want_c, want_s, d))
    assert not codes[:7].any() and not values[:7].any()


def check_product(Y, X, codes, scales, dt):
    exact, S = M.matmul(host(X), codes.cpu().numpy(), scales.cpu().numpy())
    got = host(Y)
    tol = X.shape[1] * 2.0 ** -23 * S + (2.0 ** -8 * np.abs(exact) if dt == "bf16" else 0.0)
    bad = ~(np.abs(got - exact) <= tol)
    assert np.array_equal(np.isnan(got), np.isnan(exact))
    assert not (bad & ~np.isnan(exact)).any(), float(np.nanmax(np.abs(got - exact) / np.maximum(tol, 1e-300)))


PRODUCTS = [
    # T, N, d, X, Y
    (1, 1, 1, "f32", "f32"), (1, 16, 32, "bf16", "f32"), (1, 33, 4096, "bf16", "bf16"), (2, 515, 1000, "f16", "f32"),
    (13, 250, 11008, "f32", "f32"), (16, 512, 512, "bf16", "bf16"), (17, 129, 96, "f32", "bf16"),
    (31, 4096, 288, "bf16", "bf16"), (33, 40, 40, "f32", "f32"), (64, 257, 2048, "bf16", "f32"),
    (100, 1000, 544, "bf16", "bf16"), (129, 300, 1003, "f32", "f32"), (257, 513, 160, "f16", "bf16"),
    (300, 640, 4096, "bf16", "bf16"), (1000, 777, 512, "bf16", "f32"), (513, 2305, 1056, "bf16", "bf16"),
]


@pytest.mark.parametrize("T,N,d,xdt,ydt", PRODUCTS)
def test_product(q, T, N, d, xdt, ydt):
    say(f"case product T={T} N={N} d={d} {xdt} -> {ydt}")
    W = weights(N, d, "f32", N + d).to(DEV)
    X = weights(T, d, xdt, T + d, spread=1.0).to(DEV)
    codes, scales = q.qamw_mxfp4_quantize(W)
    Y = q.qamw_mxfp4_matmul(X, codes, scales, out_dtype=DT[ydt])
    Y2 = q.qamw_mxfp4_matmul(X, codes, scales, out_dtype=DT[ydt])
    torch.cuda.synchronize()
    assert torch.equal(Y, Y2)
    check_product(Y, X, codes, scales, ydt)


@pytest.mark.parametrize("T,N,d,ydt", [
    (4001, 4090, 160, "bf16"), (4100, 4099, 72, "f32"),          # a round of the largest tiles, and one tile more
    (130, 300, 8192, "bf16"), (1000, 900, 8200, "f32"),          # few tiles, long rows: K in shares
    (1000, 2200, 1056, "bf16"), (32, 8185, 416, "f32"), (20, 600, 4000, "bf16"), (16, 8190, 640, "bf16")])
def test_product_tile_shapes(q, T, N, d, ydt):
    """Products large enough, or long enough, to take every tile shape and the splits of the contraction."""
    say(f"case tile shapes T={T} N={N} d={d} {ydt}")
    W = weights(N, d, "f32", N).to(DEV)
    X = weights(T, d, "bf16", T).to(DEV)
    codes, scales = q.qamw_mxfp4_quantize(W)
    Y = q.qamw_mxfp4_matmul(X, codes, scales, out_dtype=DT[ydt])
    Y2 = q.qamw_mxfp4_matmul(X, codes, scales, out_dtype=DT[ydt])
    torch.cuda.synchronize()
    assert torch.equal(Y, Y2)
    check_product(Y, X, codes, scales, ydt)


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_product_wide_scales(q, T):
    """Block scales over the format's range, whose products stay inside fp32."""
    say(f"case product wide scales T={T}")
    N, d = 70, 352
    rng = np.random.default_rng(T)
    block = lambda n: np.repeat(2.0 ** rng.integers(-60, 60, size=(n, d // 32)), 32, axis=1)  # noqa: E731
    W = torch.from_numpy((rng.standard_normal((N, d)) * block(N)).astype(np.float32)).to(DEV)
    X = torch.from_numpy((rng.standard_normal((T, d)) * block(T)).astype(np.float32)).to(DEV)
    codes, scales = q.qamw_mxfp4_quantize(W)
    Y = q.qamw_mxfp4_matmul(X, codes, scales)
    torch.cuda.synchronize()
    check_product(Y, X, codes, scales, "f32")


@pytest.mark.parametrize("T,N", [(1, 40), (20, 300), (150, 130)])
def test_product_nan_rows_stay_in_their_rows(q, T, N):
    say(f"case product NaN rows T={T} N={N}")
    d = 200
    W = weights(N, d, "f32", 1).to(DEV)
    X = weights(T, d, "f32", 2).to(DEV)
    W[N // 2, d - 1] = float("nan")
    W[N - 1, 0] = float("inf")
    if T > 1:
        X[T - 1, 7] = float("-inf")
    codes, scales = q.qamw_mxfp4_quantize(W)
    Y = q.qamw_mxfp4_matmul(X, codes, scales)
    torch.cuda.synchronize()
    check_product(Y, X, codes, scales, "f32")


@pytest.mark.parametrize("T,ydt", [(3, "f32"), (3, "bf16"), (150, "f32"), (150, "bf16")])
def test_product_strided(q, T, ydt):
    """X rows off 16-byte boundaries, Y rows inside a wider matrix whose rest stays."""
    say(f"case product strided T={T} {ydt}")
    N, d = 203, 333
    X = weights(T, d + 5, "bf16", 3).to(DEV)[:, 1:1 + d]
    codes, scales = q.qamw_mxfp4_quantize(weights(N, d, "f32", 4).to(DEV))
    out = torch.full((T, N + 9), -77.0, dtype=DT[ydt], device=DEV)
    q.qamw_mxfp4_matmul(X, codes, scales, out=out[:, 5:5 + N])
    torch.cuda.synchronize()
    check_product(out[:, 5:5 + N], X, codes, scales, ydt)
    assert (out[:, :5] == -77).all() and (out[:, 5 + N:] == -77).all()


def test_rotated_operands(q):
    """The codec's rotation in front of the format: (R X / s)(R W s)^T = X W^T up to the quantisation, on operands
    whose outlier channels the plain format spends its scales on."""
    T, N, d, b, seed = 64, 256, 1024, 128, 3
    rng = np.random.default_rng(8)
    r = np.where(rng.random(d) < 0.02, 30.0, 1.0)
    X = torch.from_numpy((rng.standard_normal((T, d)) * r).astype(np.float32)).to(DEV)
    W = torch.from_numpy((rng.standard_normal((N, d)) * 0.02).astype(np.float32)).to(DEV)
    exact = host(X) @ host(W).T

    def err(Xt, Wt):
        Y = q.qamw_mxfp4_matmul(Xt, *q.qamw_mxfp4_quantize(Wt))
        return float(np.linalg.norm(host(Y) - exact) / np.linalg.norm(exact))

    plain = err(X, W)
    rotated = err(q.qamw_rotate_activations(X, None, b, seed), q.qamw_rotate_activations(W, None, b, seed))
    say(f"case rotated operands: relative error {plain:.4f} plain, {rotated:.4f} rotated")
    # both operands at 4 bits with rms error about 0.11 each: 0.16; the outliers make the plain error larger
    assert rotated < 0.2 and rotated < plain


def test_no_rows(q):
    W = torch.empty(0, 64, device=DEV)
    codes, scales, values = q.qamw_mxfp4_quantize(W, values_dtype=torch.float32)
    assert codes.shape == (0, 32) and scales.shape == (0, 16) and values.shape == (0, 64)
    assert q.qamw_mxfp4_dequantize(codes, scales, 64).shape == (0, 64)
    c, s = q.qamw_mxfp4_quantize(torch.ones(3, 64, device=DEV))
    assert q.qamw_mxfp4_matmul(torch.empty(0, 64, device=DEV), c, s).shape == (0, 3)
    assert q.qamw_mxfp4_matmul(torch.ones(2, 64, device=DEV), codes, scales).shape == (2, 0)


@pytest.mark.parametrize("T", [1, 9, 48, 300])
def test_other_stream_and_graph(q, T):
    """A call on another stream, and its capture replayed several times with eager work between the replays."""
    say(f"case stream and graph T={T}")
    N, d = 520, 1024
    codes, scales = q.qamw_mxfp4_quantize(weights(N, d, "f32", 1).to(DEV))
    X = weights(T, d, "bf16", 2).to(DEV)
    want = q.qamw_mxfp4_matmul(X, codes, scales)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    q.qamw_mxfp4_matmul(X, codes, scales, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    ws = torch.empty(max(q.qamw_mxfp4_matmul_workspace_bytes(T, N, d), 256), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qamw_mxfp4_matmul(X, codes, scales, out=out, workspace=ws)
    for k in range(4):
        X.copy_(weights(T, d, "bf16", 10 + k).to(DEV))
        ws.fill_(255)
        out.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q.qamw_mxfp4_matmul(X, codes, scales))
        torch.cuda.synchronize()


def test_refusals(q):
    W = torch.ones(4, 64, device=DEV)
    codes, scales = q.qamw_mxfp4_quantize(W)
    for call in (lambda: q.qamw_mxfp4_quantize(W.double()),
                 lambda: q.qamw_mxfp4_quantize(W.cpu()),
                 lambda: q.qamw_mxfp4_quantize(W.t()),
                 lambda: q.qamw_mxfp4_quantize(W, codes=codes[:3]),
                 lambda: q.qamw_mxfp4_quantize(W, values=torch.empty(4, 63, device=DEV)),
                 lambda: q.qamw_mxfp4_dequantize(codes, scales, 65),
                 lambda: q.qamw_mxfp4_dequantize(codes, scales, 64, out_dtype=torch.float64),
                 lambda: q.qamw_mxfp4_dequantize(codes, scales, 0),
                 lambda: q.qamw_mxfp4_matmul(torch.ones(2, 65, device=DEV), codes, scales),
                 lambda: q.qamw_mxfp4_matmul(torch.ones(2, 64, device=DEV), codes, scales, out_dtype=torch.float16),
                 lambda: q.qamw_mxfp4_matmul(torch.ones(2, 64, device=DEV), codes.cpu(), scales)):
        with pytest.raises(ValueError):
            call()
    from vector_codebook_codec_amd._lib import QamwError

    with pytest.raises(QamwError):
        q.qamw_mxfp4_matmul(torch.ones(2, 64, device=DEV), codes, scales,
                            workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
