"""Calls on a stream that is not the current one: what they allocate must be
safe from work queued on the current stream before and after; needs an
MI355X.

The current stream is kept busy for about 20 ms, so that whatever a call on
the other stream does, it does first; nothing is synchronised in between."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vector_codebook_codec_amd as pkg
    from vector_codebook_codec_amd import _lib

    _lib.load()
    return pkg


@pytest.fixture(scope="module")
def busy():
    """Queues about 20 ms of work on the current stream."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(a)

    def queue():
        for _ in range(20):
            torch.mm(a, a, out=out)
    return queue


def calls(q):
    """{name: (call(stream) -> tensors, bytes of what it allocates)}"""
    rng = np.random.default_rng(3)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV)  # noqa: E731
    T, V, d, N = 192, 3000, 512, 640
    X, W, H, U = new(T, d), new(N, d) * 0.02, new(T, d), new(V, d) * 0.05
    y = torch.from_numpy(rng.integers(0, V, T)).to(DEV)
    up = torch.ones(T, device=DEV)
    codes, scales = q.qamw_mxfp4_quantize(W)
    _, lse = q.qamw_cross_entropy(H, U, y)
    r, C = torch.ones(d, device=DEV), torch.from_numpy(q.load_codebook(256)).to(DEV)
    s, sigma = q.qamw_calibrate(W, r, 0.5, 128, 7)
    packed, rn = q.qamw_encode(W, s, sigma, 128, 7, C)
    Xr = q.qamw_rotate_activations(X, s, 128, 7)
    f32 = torch.float32
    return {
        "mxfp4_quantize": (lambda st: q.qamw_mxfp4_quantize(W, values_dtype=f32, stream=st),
                           (codes.nbytes, scales.nbytes, W.nbytes)),
        "mxfp4_dequantize": (lambda st: (q.qamw_mxfp4_dequantize(codes, scales, d, stream=st),), (W.nbytes,)),
        "mxfp4_matmul": (lambda st: (q.qamw_mxfp4_matmul(X, codes, scales, stream=st),),
                         (T * N * 4, q.qamw_mxfp4_matmul_workspace_bytes(T, N, d))),
        "cross_entropy": (lambda st: q.qamw_cross_entropy(H, U, y, stream=st),
                          (T * 4, T * 4, q.qamw_cross_entropy_workspace_bytes(T, V, d, f32))),
        "cross_entropy_grad": (lambda st: q.qamw_cross_entropy_grad(H, U, y, lse, up, stream=st),
                               (H.nbytes, U.nbytes, q.qamw_cross_entropy_grad_workspace_bytes(T, V, d, f32))),
        "calibrate": (lambda st: q.qamw_calibrate(W, r, 0.5, 128, 7, stream=st),
                      (d * 4, d * 2, q.qamw_calibrate_workspace_bytes(N, d, 128))),
        "encode": (lambda st: q.qamw_encode(W, s, sigma, 128, 7, C, stream=st),
                   (packed.nbytes, rn.nbytes, q.qamw_encode_workspace_bytes(N, d))),
        "decode": (lambda st: (q.qamw_decode(packed, rn, d, s, sigma, 128, 7, C, stream=st),), (W.nbytes,)),
        "decode_matmul": (lambda st: (q.qamw_decode_matmul(Xr, packed, rn, sigma, C, stream=st),), (T * N * 4,)),
        "channel_rms": (lambda st: (q.qamw_channel_rms(X, stream=st),), (d * 4, q.qamw_channel_rms_workspace_bytes(T, d))),
    }


NAMES = ["mxfp4_quantize", "mxfp4_dequantize", "mxfp4_matmul", "cross_entropy", "cross_entropy_grad", "calibrate", "encode",
         "decode", "decode_matmul", "channel_rms"]


@pytest.fixture(scope="module")
def every(q):
    made = calls(q)
    assert sorted(made) == sorted(NAMES)
    return made


def handle_forms(side):
    return side, side.cuda_stream


@pytest.mark.parametrize("name", NAMES)
def test_blocks_that_the_current_stream_still_reads(every, busy, name):
    """Buffers of the sizes that the call allocates, freed while reads of them are queued on the current stream."""
    print(f"case queued reads {name}", flush=True)
    sys.stdout.flush()
    call, sizes = every[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    for stream in handle_forms(side):
        torch.cuda.synchronize()
        held = [torch.full((max(n, 256),), 7, dtype=torch.uint8, device=DEV) for n in sizes]
        seen = [torch.zeros_like(h) for h in held]
        torch.cuda.synchronize()
        busy()
        for s, h in zip(seen, held):
            s.copy_(h)
        del h, held
        got = call(stream)
        torch.cuda.synchronize()
        assert all((s == 7).all() for s in seen)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_results_dropped_or_reused(every, busy, name):
    """Results that the current stream still reads when they are dropped, and a second call beside that."""
    print(f"case dropped results {name}", flush=True)
    call, _ = every[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    seen = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    busy()
    for s, t in zip(seen, got):
        s.copy_(t)
    del t, got
    again = call(side)
    with torch.cuda.stream(side):
        for t in again:
            t.zero_()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(seen, want))


def test_result_dropped_before_the_stream_reads_it(q, busy):
    """lse made and read on the other stream, dropped at once; the current stream then takes blocks of its size."""
    print("case lse dropped", flush=True)
    rng = np.random.default_rng(5)
    T, V, d = 300, 2000, 256
    H = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(DEV)
    U = torch.from_numpy((rng.standard_normal((V, d)) * 0.05).astype(np.float32)).to(DEV)
    y = torch.from_numpy(rng.integers(0, V, T)).to(DEV)
    up = torch.ones(T, device=DEV)
    want = q.qamw_cross_entropy_grad(H, U, y, q.qamw_cross_entropy(H, U, y)[1], up)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
    _, lse = q.qamw_cross_entropy(H, U, y, stream=side)
    got = q.qamw_cross_entropy_grad(H, U, y, lse, up, stream=side)
    del _, lse
    for _ in range(8):
        torch.full((T,), float("nan"), device=DEV)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_default_stream_by_handle(every):
    """The null handle names the default stream, also where another one is current."""
    call, _ = every["mxfp4_matmul"]
    want = call(None)[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(0)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
