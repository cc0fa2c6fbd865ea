"""C ABI checks of the attention cache and of the adapters that need no GPU:
sizes, and refusals before anything is launched (the addresses are never
dereferenced)."""
import os

import pytest

A = 1 << 20           # 16-byte aligned
WS = 1 << 24
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -4
F32, BF16, F16 = 0, 1, 2
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    from vector_codebook_codec_amd import _lib

    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libqamw.so not built")
    return _lib.load()


def test_sizes(lib):
    for d, rb, sb in ((1, 16, 2), (32, 16, 2), (33, 32, 2), (64, 32, 2), (65, 48, 4), (128, 64, 4), (129, 80, 8), (256, 128, 8)):
        assert lib.qamw_mxfp4_cache_row_bytes(d) == rb and lib.qamw_mxfp4_cache_scale_bytes(d) == sb
    for d in (0, -1, 257, BIG):
        assert lib.qamw_mxfp4_cache_row_bytes(d) == -1 and lib.qamw_mxfp4_cache_scale_bytes(d) == -1
    need = lib.qamw_mxfp4_cache_attention_workspace_bytes
    assert need(1, 1, 1, 8, 32, 128, 1000, BF16, BF16) == 0                  # one share
    assert need(1, 1, 1, 8, 32, 128, 131072, BF16, BF16) > 0
    assert need(64, 64, 1, 8, 32, 128, 131072, BF16, BF16) > 0
    assert need(4096, 2, 2048, 8, 32, 128, 4096, BF16, BF16) > 0             # which workgroups gave up
    for bad in ((0, 1, 1, 8, 32, 128, 64, BF16, BF16), (1, 1, 1, 8, 30, 128, 64, BF16, BF16), (1, 1, 1, 8, 32, 300, 64, BF16, BF16),
                (1, 1, 1, 8, 32, 128, -1, BF16, BF16), (1, 1, 1, 8, 32, 128, 64, 3, BF16), (1, 1, 0, 8, 32, 128, 64, BF16, BF16),
                (1, BIG, 1, 8, 32, 128, 64, BF16, BF16), (BIG, 1, 1, 8, 32, 128, 64, BF16, BF16)):
        assert need(*bad) == 0, bad
    more = lib.qamw_mxfp4_adapter_matmul_workspace_bytes
    assert more(48, 4096, 4096, 16, BF16) > lib.qamw_mxfp4_matmul_workspace_bytes(48, 4096, 4096)
    for bad in ((0, 8, 64, 4, BF16), (4, 8, 64, 0, BF16), (4, 8, 64, 1025, BF16), (4, 8, 64, 4, F16)):
        assert more(*bad) == 0, bad


def write(lib, K=A, V=A, dt=BF16, T=3, heads=2, d=64, kt=128, kh=64, vt=128, vh=64, slots=A, codes=A, scales=A, pages=4, page=16):
    return lib.qamw_mxfp4_cache_write(K, V, dt, T, heads, d, kt, kh, vt, vh, slots, codes, scales, pages, page, None)


def read(lib, K=A, V=A, dt=BF16, T=3, heads=2, d=64, kt=128, kh=64, vt=128, vh=64, slots=A, codes=A, scales=A, pages=4, page=16):
    return lib.qamw_mxfp4_cache_read(codes, scales, pages, page, heads, d, slots, T, K, V, dt, kt, kh, vt, vh, None)


@pytest.mark.parametrize("call", [write, read])
def test_write_and_read_refusals(lib, call):
    for kw in (dict(codes=None), dict(scales=A + 8), dict(codes=A + 4), dict(slots=None), dict(slots=A + 4), dict(K=A + 1),
               dict(V=A + 1), dict(T=-1), dict(heads=0), dict(heads=-2), dict(d=0), dict(pages=-1), dict(kt=-1), dict(vh=-64)):
        assert call(lib, **kw) == EINVAL, kw
    for kw in (dict(dt=3), dict(d=257), dict(page=15), dict(page=24), dict(page=8), dict(page=1 << 17), dict(page=0), dict(page=-16),
               dict(heads=65537), dict(pages=BIG), dict(pages=1 << 31), dict(T=BIG), dict(T=1 << 31), dict(heads=65536, page=65536),
               dict(kt=BIG)):
        assert call(lib, **kw) == EUNSUPPORTED, kw
    assert call(lib, T=0, K=None, V=None, slots=None) == 0
    assert lib.qamw_last_error()


def test_read_may_leave_one_out_and_refuses_rows_that_overlap(lib):
    assert read(lib, K=None, V=None) == 0
    for kw in (dict(kt=64), dict(kh=63), dict(kt=127), dict(vt=0), dict(vh=0), dict(kt=64, kh=64 * 2)):
        assert read(lib, **kw) == EINVAL, kw
    assert write(lib, K=None) == EINVAL and write(lib, V=None) == EINVAL


def attend(lib, Q=A, qdt=BF16, T=6, q_heads=8, d=64, qt=512, qh=64, starts=A, sequences=2, most=3, codes=A, scales=A, pages=9,
           page=16, heads=2, table=A, cols=40, pitch=40, lengths=A, scale=0.125, causal=1, window=0, out=A, odt=BF16, ot=512, oh=64,
           lse=A, ws=WS, nbytes=1 << 30):
    return lib.qamw_mxfp4_cache_attention(Q, qdt, T, q_heads, d, qt, qh, starts, sequences, most, codes, scales, pages, page, heads,
                                          table, cols, pitch, lengths, scale, causal, window, out, odt, ot, oh, lse, ws, nbytes, None)


def test_attention_refusals(lib):
    for kw in (dict(Q=None), dict(Q=A + 1), dict(out=None), dict(out=A + 1), dict(codes=None), dict(scales=A + 1), dict(T=-1),
               dict(sequences=-1), dict(q_heads=7), dict(q_heads=0), dict(heads=0), dict(d=0), dict(most=0), dict(starts=None),
               dict(starts=A + 2), dict(table=None), dict(table=A + 1), dict(lengths=None), dict(lengths=A + 1), dict(lse=A + 2),
               dict(cols=-1), dict(pitch=39), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(window=-1), dict(ot=511), dict(oh=32), dict(qt=-1), dict(oh=0)):
        assert attend(lib, **kw) == EINVAL, kw
    for kw in (dict(qdt=5), dict(odt=-1), dict(d=300), dict(page=17), dict(cols=1 << 27, pitch=1 << 27), dict(T=BIG, ot=512),
               dict(sequences=1 << 24), dict(pages=BIG), dict(cols=BIG, pitch=BIG), dict(T=1 << 29, most=1 << 29, sequences=1 << 20),
               dict(q_heads=1 << 20)):
        assert attend(lib, **kw) == EUNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(nbytes=16)):
        assert attend(lib, cols=4000, pitch=4000, **kw) == EWORKSPACE, kw
    assert attend(lib, T=0, Q=None, out=None, lengths=None, table=None) == 0
    assert attend(lib, sequences=0, lengths=None, table=None, starts=A) == 0


def adapt(lib, X=A, xdt=BF16, T=4, d=64, ldx=64, codes=A, scales=A, N=8, a=A, b=A, n=3, rank=4, index=A, factors=None, Y=A, ydt=F32,
          ldy=8, ws=WS, nbytes=1 << 24):
    return lib.qamw_mxfp4_adapter_matmul(X, xdt, T, d, ldx, codes, scales, N, a, b, n, rank, index, factors, Y, ydt, ldy, ws, nbytes,
                                         None)


def test_adapter_refusals(lib):
    for kw in (dict(X=None), dict(X=A + 1), dict(codes=None), dict(scales=A + 4), dict(Y=None), dict(Y=A + 2), dict(ldx=63),
               dict(ldy=7), dict(T=-1), dict(N=-1), dict(d=0), dict(n=-1), dict(rank=0), dict(rank=-4), dict(a=None), dict(b=None),
               dict(a=A + 8), dict(b=A + 2), dict(index=None), dict(index=A + 2), dict(factors=A + 1)):
        assert adapt(lib, **kw) == EINVAL, kw
    for kw in (dict(xdt=F16), dict(ydt=F16), dict(rank=1025), dict(n=1 << 40), dict(T=BIG), dict(N=BIG, ldy=BIG), dict(d=BIG, ldx=BIG),
               dict(n=1 << 30, rank=1024, d=1 << 20, ldx=1 << 20)):
        assert adapt(lib, **kw) == EUNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=WS + 8), dict(nbytes=64)):
        assert adapt(lib, **kw) == EWORKSPACE, kw
    assert adapt(lib, T=0, X=None, Y=None, ws=None) == 0 and adapt(lib, N=0, ldy=0, codes=None, scales=None, Y=None, ws=None) == 0
