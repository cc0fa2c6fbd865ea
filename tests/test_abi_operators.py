"""C ABI checks of the 4-bit operators and of the cross entropy that need no
GPU: host helpers, and refusals before anything is launched (the addresses
are never dereferenced)."""
import os

import pytest

A = 1 << 20           # 16-byte aligned
WS = 1 << 24
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -4
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from vector_codebook_codec_amd import _lib

    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libqamw.so not built")
    return _lib.load()


def test_sizes(lib):
    for d, rb, sb in ((1, 16, 16), (32, 16, 16), (33, 32, 16), (512, 256, 16), (513, 272, 32), (11008, 5504, 352)):
        assert lib.qamw_mxfp4_row_bytes(d) == rb and lib.qamw_mxfp4_scale_bytes(d) == sb
    for d in (0, -1, (1 << 20) + 1):
        assert lib.qamw_mxfp4_row_bytes(d) == -1 and lib.qamw_mxfp4_scale_bytes(d) == -1
    assert lib.qamw_mxfp4_matmul_workspace_bytes(0, 16, 64) == 0
    # at least the quantised activations
    assert lib.qamw_mxfp4_matmul_workspace_bytes(7, 16, 4096) >= 7 * (2048 + 128)
    assert lib.qamw_cross_entropy_workspace_bytes(0, 100, 64, BF16) == 0
    assert lib.qamw_cross_entropy_workspace_bytes(5, 100, 64, F16) == 0
    assert lib.qamw_cross_entropy_workspace_bytes(5, 100, 64, BF16) > 0
    # far less than the logits of a large vocabulary
    assert lib.qamw_cross_entropy_workspace_bytes(4096, 131072, 4096, BF16) < 4096 * 131072 * 4 // 16
    assert lib.qamw_cross_entropy_grad_workspace_bytes(4096, 131072, 4096, BF16) < 4096 * 131072 * 4 // 2
    assert lib.qamw_cross_entropy_grad_workspace_bytes(4096, 131072, 4096, F32) > 0


def quantize(lib, W=A, wdt=BF16, N=8, d=64, ldw=64, codes=A, scales=A, values=None, vdt=BF16, ldv=64):
    return lib.qamw_mxfp4_quantize(W, wdt, N, d, ldw, codes, scales, values, vdt, ldv, None)


def test_quantize_refusals(lib):
    for kw in (dict(W=None), dict(W=A + 1), dict(codes=None), dict(scales=None), dict(codes=A + 8), dict(scales=A + 8),
               dict(N=-1), dict(d=0), dict(ldw=63), dict(values=A + 1), dict(values=A, ldv=63)):
        assert quantize(lib, **kw) == EINVAL, kw
    for kw in (dict(wdt=3), dict(wdt=-1), dict(values=A, vdt=7), dict(d=(1 << 20) + 1, ldw=1 << 21)):
        assert quantize(lib, **kw) == EUNSUPPORTED, kw
    assert quantize(lib, N=0, W=None, codes=None, scales=None) == 0
    assert b"" != lib.qamw_last_error()


def test_dequantize_refusals(lib):
    def call(codes=A, scales=A, N=8, d=64, out=A, dt=BF16, ldo=64):
        return lib.qamw_mxfp4_dequantize(codes, scales, N, d, out, dt, ldo, None)

    for kw in (dict(codes=None), dict(scales=A + 1), dict(out=None), dict(out=A + 1), dict(ldo=32), dict(d=-3), dict(N=-1)):
        assert call(**kw) == EINVAL, kw
    assert call(dt=5) == EUNSUPPORTED
    assert call(N=0, codes=None, scales=None, out=None) == 0


def test_matmul_refusals(lib):
    def call(X=A, xdt=BF16, T=4, d=64, ldx=64, codes=A, scales=A, N=8, Y=A, ydt=F32, ldy=8, ws=WS, nbytes=1 << 20):
        return lib.qamw_mxfp4_matmul(X, xdt, T, d, ldx, codes, scales, N, Y, ydt, ldy, ws, nbytes, None)

    for kw in (dict(X=None), dict(X=A + 1), dict(codes=None), dict(scales=None), dict(Y=None), dict(Y=A + 2), dict(ldx=8),
               dict(ldy=7), dict(T=-1), dict(N=-1), dict(d=0)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(xdt=4), dict(ydt=F16), dict(T=1 << 32)):
        assert call(**kw) == EUNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(nbytes=16)):
        assert call(**kw) == EWORKSPACE, kw
    assert call(T=0, X=None, Y=None, ws=None) == 0 and call(N=0, ldy=0, codes=None, scales=None, Y=None, ws=None) == 0


def test_cross_entropy_refusals(lib):
    def call(H=A, dt=BF16, T=4, d=64, ldh=64, W=A, V=100, ldw=64, y=A, loss=A, lse=A, ws=WS, nbytes=1 << 24):
        return lib.qamw_cross_entropy(H, dt, T, d, ldh, W, V, ldw, y, loss, lse, ws, nbytes, None)

    for kw in (dict(H=None), dict(H=A + 8), dict(W=None), dict(W=A + 8), dict(y=None), dict(y=A + 4), dict(loss=None),
               dict(lse=None), dict(lse=A + 2), dict(ldh=60), dict(ldw=68), dict(d=60), dict(T=-1), dict(V=0), dict(d=0)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(dt=F16), dict(dt=9), dict(d=1 << 22, ldh=1 << 22, ldw=1 << 22), dict(T=1 << 22), dict(ldw=1 << 22),
               dict(V=1 << 31)):
        assert call(**kw) == EUNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=WS + 8), dict(nbytes=8)):
        assert call(**kw) == EWORKSPACE, kw
    assert call(T=0, H=None, y=None, loss=None, lse=None, ws=None) == 0


def test_cross_entropy_grad_refusals(lib):
    def call(H=A, dt=BF16, T=4, d=64, ldh=64, W=A, V=100, ldw=64, y=A, lse=A, dloss=A, dH=A, lddh=64, dW=A, lddw=64, ws=WS,
             nbytes=1 << 28):
        return lib.qamw_cross_entropy_grad(H, dt, T, d, ldh, W, V, ldw, y, lse, dloss, dH, lddh, dW, lddw, ws, nbytes, None)

    for kw in (dict(H=None), dict(W=A + 8), dict(y=None), dict(lse=None), dict(dloss=None), dict(dH=A + 8), dict(dW=A + 8),
               dict(lddh=63), dict(lddw=63), dict(lddw=68), dict(d=60)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(dt=F16), dict(T=1 << 22)):
        assert call(**kw) == EUNSUPPORTED, kw
    for kw in (dict(ws=None), dict(nbytes=8)):
        assert call(**kw) == EWORKSPACE, kw
    assert call(dH=None, dW=None, ws=None) == 0
