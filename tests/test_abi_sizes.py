"""Sizes and leading dimensions near the ends of 64 bits: refused on the host
before anything is multiplied with them.  Needs no GPU; the addresses are
never dereferenced."""
import os

import pytest

A, WS = 1 << 20, 1 << 24
EINVAL, EUNSUPPORTED = -1, -2
F32, BF16 = 0, 1
HUGE = [1 << 61, 1 << 62, (1 << 62) + 64, (1 << 63) - 64]        # multiples of 64


@pytest.fixture(scope="module")
def lib():
    from vector_codebook_codec_amd import _lib

    if not os.path.exists(os.environ.get("QAMW_LIBRARY", _lib.LIB_PATH)):
        pytest.skip("libqamw.so not built")
    return _lib.load()


def forward(lib, dt, T=4, d=64, V=100, ldh=64, ldw=64):
    return lib.qamw_cross_entropy(A, dt, T, d, ldh, A, V, ldw, A, A, A, WS, 1 << 40, None)


def gradient(lib, dt, T=4, d=64, V=100, ldh=64, ldw=64, lddh=64, lddw=64):
    return lib.qamw_cross_entropy_grad(A, dt, T, d, ldh, A, V, ldw, A, A, A, A, lddh, A, lddw, WS, 1 << 40, None)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", HUGE)
def test_cross_entropy_huge_sizes(lib, n, dt):
    for call in (forward, gradient):
        assert call(lib, dt, d=n, ldh=n, ldw=n) == EUNSUPPORTED
        assert call(lib, dt, d=n) == EUNSUPPORTED
        assert call(lib, dt, T=n) == EUNSUPPORTED
        assert call(lib, dt, V=n) == EUNSUPPORTED
        assert call(lib, dt, ldh=n) == EUNSUPPORTED
        assert call(lib, dt, ldw=n) == EUNSUPPORTED
    for size in (lib.qamw_cross_entropy_workspace_bytes, lib.qamw_cross_entropy_grad_workspace_bytes):
        assert size(4, 100, n, dt) == 0 and size(n, 100, 64, dt) == 0 and size(4, n, 64, dt) == 0


@pytest.mark.parametrize("dt,most", [(F32, 1 << 20), (BF16, 1 << 21)])
def test_cross_entropy_first_size_refused(lib, dt, most):
    """Rows of H and W, and a row of T elements, stay under 4 MiB; a leading dimension may be 4 MiB."""
    size = lib.qamw_cross_entropy_grad_workspace_bytes
    assert size(most, 8, 8, dt) == 0 and size(most - 1, 8, 8, dt) > 0
    assert size(1, 8, most, dt) == 0 and size(1, 8, most - 8, dt) > 0
    assert forward(lib, dt, T=most) == EUNSUPPORTED and forward(lib, dt, d=most, ldh=most, ldw=most) == EUNSUPPORTED
    assert forward(lib, dt, ldh=most + 8) == EUNSUPPORTED and forward(lib, dt, ldw=most + 8) == EUNSUPPORTED


@pytest.mark.parametrize("n", HUGE)
def test_leading_dimensions_off_16_bytes(lib, n):
    """The alignment of a row is that of its leading dimension, whatever the number of bytes wraps to."""
    for dt, off in ((F32, 1), (F32, 2), (BF16, 4), (BF16, 1)):
        assert gradient(lib, dt, lddh=n + off) == EINVAL and gradient(lib, dt, lddw=n + off) == EINVAL
        assert lib.qamw_channel_rms(A, dt, 8, 64, n + off, A, WS, 1 << 30, None) == EINVAL
        assert lib.qamw_rotate_activations(A, dt, 8, 64, n + off, None, 64, 0, A, 64, None) == EINVAL


@pytest.mark.parametrize("n", HUGE)
def test_mxfp4_huge_sizes(lib, n):
    assert lib.qamw_mxfp4_row_bytes(n) == -1 and lib.qamw_mxfp4_scale_bytes(n) == -1
    assert lib.qamw_mxfp4_quantize(A, BF16, 8, n, n, A, A, None, 0, 0, None) == EUNSUPPORTED
    assert lib.qamw_mxfp4_quantize(A, BF16, n, 64, 64, A, A, None, 0, 0, None) == EUNSUPPORTED
    assert lib.qamw_mxfp4_dequantize(A, A, n, 64, A, BF16, 64, None) == EUNSUPPORTED
    assert lib.qamw_mxfp4_matmul(A, BF16, n, 64, 64, A, A, 8, A, F32, 8, WS, 1 << 40, None) == EUNSUPPORTED
    assert lib.qamw_mxfp4_matmul(A, BF16, 4, 64, 64, A, A, n, A, F32, n, WS, 1 << 40, None) == EUNSUPPORTED
    assert lib.qamw_mxfp4_matmul_workspace_bytes(n, 8, 64) == 0 and lib.qamw_mxfp4_matmul_workspace_bytes(8, n, 64) == 0


@pytest.mark.parametrize("dt", [F32, BF16])
def test_cross_entropy_more_workgroups_than_a_launch_holds(lib, dt):
    """A launch has fewer than 2^32 threads: heads of 2^27 rows for a few tokens, 2^39 logits for many."""
    size = lib.qamw_cross_entropy_workspace_bytes
    for T in (1, 4):
        assert size(T, 1 << 27, 8, dt) == 0 and size(T, (1 << 27) - 16, 8, dt) > 0
        assert forward(lib, dt, T=T, V=1 << 27) == EUNSUPPORTED and gradient(lib, dt, T=T, V=1 << 27) == EUNSUPPORTED
    T = (1 << 20) - 8                                    # 2^13 or 2^12 tiles of tokens
    V = 1 << (18 if dt == F32 else 19)                   # in fp32 128 x 128 tiles, in bf16 256 x 256
    assert size(T, V, 512, dt) == 0 and size(T, V // 16, 512, dt) > 0
    assert forward(lib, dt, T=T, V=V) == EUNSUPPORTED


def test_mxfp4_more_workgroups_than_a_launch_holds(lib):
    def call(T, N):
        return lib.qamw_mxfp4_matmul(A, BF16, T, 64, 64, A, A, N, A, F32, N, WS, 16, None)

    EWORKSPACE = -4
    assert call(1, 1 << 27) == EUNSUPPORTED and call(1, (1 << 27) - 16) == EWORKSPACE
    assert call(16, 1 << 31) == EUNSUPPORTED
    assert call(1 << 31, 64) == EUNSUPPORTED and call(1 << 29, 64) == EWORKSPACE       # 2^25 and 2^23 tiles of 64 x 64
    assert call(1 << 20, 1 << 19) == EUNSUPPORTED and call(1 << 20, 1 << 18) == EWORKSPACE
