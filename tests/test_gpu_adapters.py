"""GPU parity of the 4-bit product with low-rank adapters against the oracle
(oracle/mxfp4.py); needs an MI355X.

Criteria, element by element:
  * the shared product as in test_gpu_mxfp4.py: d 2^-23 S, S the sum of its
    products' magnitudes;
  * the adapters: sums of d and of r fp32 products, rounded to at most 2^-23 of
    S2 = |f| sum_k |B| sum_j |A| |X| each time, and the factor: (d + r + 2)
    2^-23 S2; U as bf16 numbers is off by 2^-16 of each entry for a bf16 result
    (two of them), 2^-24 for fp32 (three): times sum_k |U| |B|, for bf16;
  * the sum of both: 2^-23 (S + S2), and the result's half step, 2^-8 for bf16;
over all elements, where there are 256 or more, in the root mean square: 2e-3 for bf16 results, 1e-5 for fp32.
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
        bound += (2.0 ** -16 if out == "bf16" else 2.0 ** -24) * inner
    if out == "bf16":
        bound += 2.0 ** -8 * np.abs(want)
    off = np.abs(got - want)
    assert (off <= bound).all(), (off / np.maximum(bound, 1e-300)).max()
    most = 2e-3 if out == "bf16" else 1e-5
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


@pytest.mark.parametrize("T,N,d,r,how", [(1, 300, 64, 16, "each"), (12, 300, 96, 20, "each"), (24, 700, 64, 16, "each"), (70, 200, 128, 33, "each"),
                                         (300, 520, 128, 16, "runs"), (600, 700, 256, 64, "runs"), (600, 300, 100, 72, "each"),
                                         (513, 4200, 64, 136, "runs")])
def test_other_tokens_do_not_matter(q, T, N, d, r, how):
    """Infinities and NaN in an adapter, its factor and its tokens stay with the tokens that use it."""
    say(f"case apart T={T} N={N} d={d} r={r} {how}")
    n = 5
    for dt in ("bf16", "f32"):
        rng, X, codes, scales, A, B, f = make(q, T, N, d, r, n, dt, T + N)
        index = choose(rng, T, n, how)
        bad = (index == 2) | (index == 4)
        i = torch.from_numpy(index).to(DEV)
        clean = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, i, f, out_dtype=DT[dt])
        A[2], B[2], f[4] = float("nan"), float("inf"), float("inf")
        X[torch.from_numpy(index == 2).to(DEV)] = float("nan")
        got = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, i, f, out_dtype=DT[dt])
        torch.cuda.synchronize()
        keep = torch.from_numpy(~bad)
        assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
        assert not torch.isfinite(got.cpu()[torch.from_numpy(index == 2)]).any()


@pytest.mark.parametrize("T,N,d,r,n", [(4000, 300, 512, 16, 5), (2049, 5000, 264, 40, 60), (1025, 300, 1000, 128, 3)])
def test_many_tokens(q, T, N, d, r, n):
    for dt, out in (("bf16", "bf16"), ("bf16", "f32")):
        say(f"case many tokens T={T} N={N} d={d} r={r} n={n} {out}")
        rng, X, codes, scales, A, B, f = make(q, T, N, d, r, n, dt, T)
        index = choose(rng, T, n, "runs")
        wide = torch.full((T, d + 8), float("nan"), dtype=DT[dt], device=DEV)
        wide[:, :d] = X
        got = q.qamw_mxfp4_adapter_matmul(wide[:, :d], codes, scales, A, B, torch.from_numpy(index).to(DEV), f, out_dtype=DT[out])
        torch.cuda.synchronize()
        check(got, X, codes, scales, A, B, index, f, dt, out)


def test_no_factors_and_no_adapters(q):
    say("case no factors")
    for T in (3, 20, 100, 300):
        rng, X, codes, scales, A, B, f = make(q, T, 200, 96, 8, 3, "bf16", T)
        index = torch.from_numpy(choose(rng, T, 3, "each")).to(DEV)
        got = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, index)
        ones = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, index, torch.ones(3, device=DEV))
        none = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A[:0], B[:0], index)
        base = q.qamw_mxfp4_matmul(X, codes, scales)
        torch.cuda.synchronize()
        assert torch.equal(got, ones) and torch.equal(none, base)


def test_adapters_in_a_graph(q):
    """Captured once, replayed with other tokens and adapters, eager calls in between."""
    say("case graph")
    for T in (2, 24, 60, 400):
        rng, X, codes, scales, A, B, f = make(q, T, 520, 256, 16, 6, "bf16", T)
        index = torch.from_numpy(choose(rng, T, 6, "each")).to(DEV)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, index, f)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, index, f)
        for _ in range(4):
            X.copy_(torch.randn_like(X))
            index.copy_(torch.from_numpy(choose(rng, T, 6, "each")))
            want = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, index, f)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_adapter_refusals(q):
    rng, X, codes, scales, A, B, f = make(q, 5, 40, 64, 4, 2, "bf16", 1)
    index = torch.zeros(5, dtype=torch.int32, device=DEV)
    for kw in (dict(X=X.half()), dict(X=X.cpu()), dict(A=A.float()), dict(B=B[:, :-1]), dict(A=A.transpose(1, 2)), dict(A=A[0]),
               dict(index=index.long()), dict(index=index[:4]), dict(factors=f[:1]), dict(factors=f.double()), dict(out=X),
               dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            q.qamw_mxfp4_adapter_matmul(**{**dict(X=X, codes=codes, scales=scales, A=A, B=B, index=index, factors=f), **kw})


def test_serving_step(q):
    """One layer of a serving step as its parts are used together: projections in 4 bits with the requests' adapters, the
    cache's write, attention over it, the output projection; against the same in 64 bits from the 4-bit values."""
    say("case serving step")
    from oracle import mxfp4_cache as C

    heads, group, hd, page, d, r = 2, 4, 64, 16, 256, 8
    rng = np.random.default_rng(11)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    seqs = [(5, 5), (9, 9), (1, 1)]
    T = sum(n for n, _ in seqs)
    N = (heads * group + 2 * heads) * hd
    Wq = [q.qamw_mxfp4_quantize((new(n, k) * k ** -0.5).to(DEV)) for n, k in ((N, d), (d, heads * group * hd))]
    A, B = (new(2, r, d) * d ** -0.5).to(DEV), (new(2, N, r) * 0.3).to(DEV)
    index = np.repeat(np.array([1, -1, 0], dtype=np.int32), [5, 9, 1])
    codes, scales = q.qamw_mxfp4_cache_new(6, heads, page, hd)
    table = torch.tensor([[4], [1], [2]], dtype=torch.int32, device=DEV)
    slots = torch.cat([torch.arange(n) + 16 * p for (n, _), p in zip(seqs, (4, 1, 2))]).to(DEV)
    X = new(T, d).to(DEV)
    qkv = q.qamw_mxfp4_adapter_matmul(X, *Wq[0], A, B, torch.from_numpy(index).to(DEV))
    Q, K, V = (t.view(T, -1, hd) for t in qkv.split([heads * group * hd, heads * hd, heads * hd], dim=1))
    q.qamw_mxfp4_cache_write(K, V, slots, codes, scales)
    starts = torch.tensor([0, 5, 14, 15], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([5, 9, 1], dtype=torch.int32, device=DEV)
    out, _ = q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, 9)
    Y = q.qamw_mxfp4_matmul(out.reshape(T, -1), *Wq[1])
    torch.cuda.synchronize()
    h = [tuple(t.cpu().numpy() for t in w) for w in Wq]
    want = M.adapter_matmul(host(X), *h[0], host(A), host(B), index, np.ones(2))[0]
    # the cache holds what these very projections round to; from there on everything is compared
    assert np.linalg.norm(host(qkv) - want) <= 1e-5 * np.linalg.norm(want)
    c, s = C.new(6, heads, page, hd)
    C.write(c, s, host(K), host(V), slots.tolist())
    assert np.array_equal(c, codes.cpu().numpy()) and np.array_equal(s, scales.cpu().numpy())
    o = C.attention(host(Q), c, s, table.cpu().numpy(), [5, 9, 1], [0, 5, 14, 15], float(np.float32(hd ** -0.5)))[0]
    assert np.linalg.norm(host(out) - o) <= 1e-5 * np.linalg.norm(o)
    y, _ = M.matmul(host(out).reshape(T, -1), *h[1])
    assert np.linalg.norm(host(Y) - y) <= 1e-5 * np.linalg.norm(y)


@pytest.mark.parametrize("T", [3, 60, 400])
def test_on_another_stream(q, T):
    """Results and workspaces of calls on a stream that is not the current one, which is busy."""
    say(f"case stream T={T}")
    rng, X, codes, scales, A, B, f = make(q, T, 520, 256, 16, 6, "bf16", T)
    index = torch.from_numpy(choose(rng, T, 6, "each")).to(DEV)
    want = q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, index, f).clone()
    a = torch.ones(4096, 4096, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a @ a
    got = [q.qamw_mxfp4_adapter_matmul(X, codes, scales, A, B, index, f, stream=s) for s in (side, side.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
