"""GPU parity of the vocabulary cross entropy and its gradient against the
oracle (oracle/cross_entropy.py); needs an MI355X.

Tolerances, from the arithmetic (u = 2^-24, S = sum of the products'
magnitudes of one logit, e = its largest over a token's logits):
  * a logit: fp32 accumulation of d products, each partial sum rounded to at
    most 2^-23 S:  dz = d 2^-23 e
  * exp: the argument z - m (|z - m| <= 90 where the result counts) is rounded
    three times: relative error 300 u; sums of them along a fixed tree of at
    most 600 additions in a row: 600 u; log of the sum and the last additions:
    (|lse| + 4) 2u.  loss and lse: dz + dz + 1000 u + (|lse| + 4) 2u
  * G: relative error dp = loss's error + dz + 400 u of p, plus u; bf16: G
    itself rounded, 2^-9
  * dH, dW: the sum of |G| error times the other factor, fp32 accumulation of
    K terms (K 2^-23 of the sum of magnitudes); bf16: 2^-8 of the result.
"""
import sys

import numpy as np
import pytest

from oracle import cross_entropy as C

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


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


def make(T, V, d, dt, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    W = torch.from_numpy((rng.standard_normal((V, d)) * scale / np.sqrt(d)).astype(np.float32)).to(DT[dt])
    H = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32) * 2).to(DT[dt])
    y = rng.integers(0, V, size=T)
    y[rng.random(T) < 0.15] = -100
    if T > 3:
        y[1], y[2], y[3] = V, -1, V - 1               # first index past the end, a negative one, the last one
    g = rng.standard_normal(T).astype(np.float32)
    return H.to(DEV), W.to(DEV), torch.from_numpy(y).to(DEV), torch.from_numpy(g).to(DEV)


def loss_tolerance(H, W, lse):
    d = H.shape[1]
    dz = d * 2.0 ** -23 * (np.abs(host(H)) @ np.abs(host(W)).T).max(axis=1, initial=0)
    return dz, 2 * dz + 1000 * U + (np.abs(lse) + 4) * 2 * U


def check_loss(loss, lse, H, W, y):
    want, want_lse = C.forward(host(H), host(W), host(y).astype(np.int64))
    _, tol = loss_tolerance(H, W, want_lse)
    assert (np.abs(host(lse) - want_lse) <= tol).all()
    assert (np.abs(host(loss) - want) <= tol).all()
    assert (host(loss)[~C.counted(y.cpu().numpy(), W.shape[0])] == 0).all()


def check_grad(dH, dW, H, W, y, g, dt):
    Hh, Wh, yh, gh = host(H), host(W), y.cpu().numpy(), host(g)
    on = C.counted(yh, Wh.shape[0])
    _, lse = C.forward(np.where(on[:, None], Hh, 0), Wh, yh)
    Hz = np.where(on[:, None], Hh, 0.0)
    dz = Hh.shape[1] * 2.0 ** -23 * (np.abs(Hz) @ np.abs(Wh).T).max(axis=1, initial=0)
    dp = 3 * dz + 1400 * U + (np.abs(lse) + 4) * 2 * U
    G = C.logit_grad(Hz, Wh, yh, gh)
    p = np.abs(G)
    for t in np.nonzero(on)[0]:
        p[t, yh[t]] = abs(gh[t]) * abs(G[t, yh[t]] / gh[t] + 1) if gh[t] else 0.0
    dG = p * dp[:, None] + np.abs(G) * (2.0 ** -8 if dt == "bf16" else 4 * U)
    out = 2.0 ** -8 if dt == "bf16" else 2 * U
    for got, want, tol in ((dH, G @ Wh, dG @ np.abs(Wh) + Wh.shape[0] * 2.0 ** -23 * (np.abs(G) @ np.abs(Wh))),
                           (dW, G.T @ Hz, dG.T @ np.abs(Hz) + Hz.shape[0] * 2.0 ** -23 * (np.abs(G).T @ np.abs(Hz)))):
        if got is None:
            continue
        over = np.abs(host(got) - want) - (tol + out * np.abs(want) + 1e-37)
        assert not (~(over <= 0)).any(), float(np.nanmax(over))
    if dH is not None:
        assert not host(dH)[~on].any()


CASES = [
    # T, V, d, dtype, spread of the logits
    (1, 1, 8, "f32", 1.0), (1, 2, 8, "bf16", 1.0), (1, 257, 72, "bf16", 1.0), (1, 5003, 512, "bf16", 3.0),
    (2, 130, 16, "f32", 1.0), (5, 1003, 4096, "bf16", 2.0), (16, 128, 64, "bf16", 1.0), (17, 129, 40, "f32", 4.0),
    (33, 640, 136, "bf16", 1.0), (127, 255, 128, "f32", 1.0), (130, 300, 1000, "bf16", 1.0), (257, 1025, 264, "bf16", 6.0),
    (300, 5003, 512, "f32", 1.0), (300, 5003, 512, "bf16", 1.0), (520, 2050, 96, "bf16", 1.0), (8, 20000, 32, "bf16", 1.0),
]


@pytest.mark.parametrize("T,V,d,dt,scale", CASES)
def test_loss_and_gradient(q, T, V, d, dt, scale):
    say(f"case loss and gradient T={T} V={V} d={d} {dt}")
    H, W, y, g = make(T, V, d, dt, T * 7 + V, scale)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    loss2, lse2 = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    dH2, dW2 = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dH, dH2) and torch.equal(dW, dW2)
    check_loss(loss, lse, H, W, y)
    check_grad(dH, dW, H, W, y, g, dt)


@pytest.mark.parametrize("T,V,d,dt", [
    (4001, 4100, 64, "bf16"), (4001, 4090, 64, "bf16"), (4001, 4090, 32, "f32"),   # logits in the largest tiles
    (4090, 300, 4096, "bf16"), (2050, 200, 2048, "f32"),         # dH in the largest tiles
    (64, 4090, 4096, "bf16"), (32, 4090, 4096, "f32"),           # dW in the largest tiles
    (64, 4100, 4096, "bf16"), (1030, 1500, 1032, "bf16"),        # middle ones
    (3, 2100, 2048, "bf16"), (16, 1100, 4096, "bf16"), (7, 4200, 520, "f32")])   # few tokens, a head over 8 MB
def test_tile_shapes(q, T, V, d, dt):
    """Sizes that take every tile shape and the few-token form in the logits and in both products."""
    say(f"case tile shapes T={T} V={V} d={d} {dt}")
    H, W, y, g = make(T, V, d, dt, T + V)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    dH2, dW2 = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    assert torch.equal(dH, dH2) and torch.equal(dW, dW2)
    check_loss(loss, lse, H, W, y)
    check_grad(dH, dW, H, W, y, g, dt)


@pytest.mark.parametrize("T", [3, 16])
def test_few_tokens_masks_and_strides(q, T):
    """The few-token form: hidden states that are not counted hold NaN, operands and gradients are column ranges of
    wider matrices, and the gradients come alone too."""
    say(f"case few tokens T={T}")
    V, d = 3000, 2048
    H, W, y, g = make(T, V, d + 24, "bf16", 30 + T)
    H, W = H[:, 8:8 + d], W[:, 16:16 + d]
    y[0], y[T - 1], y[1] = 5, -7, 5
    H[T - 1] = float("nan")
    g[T - 1] = float("inf")
    big_h = torch.full((T, d + 16), -77.0, dtype=torch.bfloat16, device=DEV)
    big_w = torch.full((V, d + 32), -77.0, dtype=torch.bfloat16, device=DEV)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    q.qamw_cross_entropy_grad(H, W, y, lse, g, dH=big_h[:, 8:8 + d], dW=big_w[:, 16:16 + d])
    dH, _ = q.qamw_cross_entropy_grad(H, W, y, lse, g, need_dW=False)
    _, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g, need_dH=False)
    torch.cuda.synchronize()
    assert torch.equal(dH, big_h[:, 8:8 + d]) and torch.equal(dW, big_w[:, 16:16 + d])
    check_grad(dH, dW, H, W, y, g, "bf16")
    for b, o in ((big_h, 8), (big_w, 16)):
        assert (b[:, :o] == -77).all() and (b[:, o + d:] == -77).all()


@pytest.mark.parametrize("scale", [1e-30, 1.0 / 3686, 1e20])
def test_upstream_scale(q, scale):
    """Upstream gradients far from 1, all the same or not: G is kept relative to the largest."""
    say(f"case upstream scale {scale}")
    H, W, y, g = make(90, 400, 64, "bf16", 21)
    _, lse = q.qamw_cross_entropy(H, W, y)
    for up in (torch.full_like(g, scale), g * scale):
        dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, up)
        torch.cuda.synchronize()
        check_grad(dH, dW, H, W, y, up, "bf16")
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, torch.zeros_like(g))
    torch.cuda.synchronize()
    assert not dH.any() and not dW.any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_gradient_alone(q, dt):
    H, W, y, g = make(70, 333, 96, dt, 4)
    _, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    a, none = q.qamw_cross_entropy_grad(H, W, y, lse, g, need_dW=False)
    none2, b = q.qamw_cross_entropy_grad(H, W, y, lse, g, need_dH=False)
    torch.cuda.synchronize()
    assert none is None and none2 is None and torch.equal(a, dH) and torch.equal(b, dW)
    assert q.qamw_cross_entropy_grad(H, W, y, lse, g, need_dH=False, need_dW=False) == (None, None)


@pytest.mark.parametrize("T,dt", [(3, "bf16"), (140, "bf16"), (140, "f32")])
def test_uncounted_tokens(q, T, dt):
    """NaN and infinities in the hidden states of tokens that are not counted reach nothing; with no token counted all
    gradients are 0."""
    say(f"case uncounted tokens T={T} {dt}")
    H, W, y, g = make(T, 300, 64, dt, 6)
    y[0], y[T - 1] = -100, 2 ** 40
    H[0] = float("nan")
    H[T - 1, 5] = float("inf")
    g[0] = float("nan")
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    assert loss[0] == 0 and loss[T - 1] == 0 and torch.isnan(lse[0])
    check_grad(dH, dW, H, W, y, g, dt)
    y.fill_(-100)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    assert not loss.any() and not dH.any() and not dW.any()


def test_nan_of_a_counted_token_stays_in_its_row(q):
    H, W, y, g = make(40, 200, 32, "f32", 7)
    y[:] = 5
    H[9, 1] = float("nan")
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    keep = torch.arange(40, device=DEV) != 9
    assert torch.isnan(loss[9]) and torch.isfinite(loss[keep]).all()
    assert torch.isnan(dH[9]).all() and torch.isfinite(dH[keep]).all() and torch.isnan(dW).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_extreme_logits(q, dt):
    """Logits of +-1e4 (far past exp's range) and a token whose target holds all the mass."""
    say(f"case extreme logits {dt}")
    H, W, y, g = make(6, 500, 16, dt, 8, scale=1.0)
    H[0] *= 4000.0
    H[1] *= -4000.0
    H[4] = W[7] * 1000
    y[:2] = 3
    y[4] = 7
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    check_loss(loss, lse, H, W, y)
    assert torch.isfinite(dH).all() and torch.isfinite(dW).all()


def test_gradient_against_differences(q):
    """The fp32 kernel's gradient along random directions against central differences of the 64-bit loss."""
    T, V, d = 37, 211, 48
    H, W, y, g = make(T, V, d, "f32", 12)
    _, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    yh, gh = y.cpu().numpy(), host(g)
    up = np.where(C.counted(yh, V), gh, 0.0)
    total = lambda a, b: float(C.forward(a, b, yh)[0] @ up)  # noqa: E731
    rng = np.random.default_rng(1)
    h = 1e-4
    for _ in range(4):
        A, B = rng.standard_normal((T, d)), rng.standard_normal((V, d))
        num = (total(host(H) + h * A, host(W)) - total(host(H) - h * A, host(W))) / (2 * h)
        ana = float((host(dH) * A).sum())
        # truncation h^2/6 times a third derivative of order T |A|^3 (below 1e4): 2e-5; fp32 gradients: 1e-5 of the sum
        assert abs(num - ana) <= 1e-4 + 1e-5 * float(np.abs(host(dH) * A).sum())
        num = (total(host(H), host(W) + h * B) - total(host(H), host(W) - h * B)) / (2 * h)
        ana = float((host(dW) * B).sum())
        assert abs(num - ana) <= 1e-2 * h + 1e-3 + 1e-5 * float(np.abs(host(dW) * B).sum())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strided_operands(q, dt):
    """H, W and the gradients as column ranges of wider matrices, whose rest stays."""
    say(f"case strided {dt}")
    T, V, d = 45, 170, 72
    H, W, y, g = make(T, V, d + 24, dt, 9)
    H, W = H[:, 8:8 + d], W[:, 16:16 + d]
    big_h = torch.full((T, d + 16), -77.0, dtype=DT[dt], device=DEV)
    big_w = torch.full((V, d + 32), -77.0, dtype=DT[dt], device=DEV)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    q.qamw_cross_entropy_grad(H, W, y, lse, g, dH=big_h[:, 8:8 + d], dW=big_w[:, 16:16 + d])
    torch.cuda.synchronize()
    check_loss(loss, lse, H, W, y)
    check_grad(big_h[:, 8:8 + d], big_w[:, 16:16 + d], H, W, y, g, dt)
    for b, o in ((big_h, 8), (big_w, 16)):
        assert (b[:, :o] == -77).all() and (b[:, o + d:] == -77).all()


@pytest.mark.parametrize("T,V,d", [(9, 40000, 4096), (700, 90000, 256)])
def test_many_pieces(q, T, V, d):
    """Vocabularies that the gradient walks in more than one piece or that fill many tiles, the last one partly."""
    say(f"case many pieces T={T} V={V} d={d}")
    H, W, y, g = make(T, V, d, "bf16", 10)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    check_loss(loss, lse, H, W, y)
    check_grad(dH, dW, H, W, y, g, "bf16")


def test_head_past_32_bit_offsets(q):
    """A head of 2.2e9 elements; the counted targets are in its last rows."""
    T, V, d = 3, 265000, 8192
    say(f"case head past 32-bit offsets {V} x {d}")
    W = torch.zeros(V, d, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(2)
    last = torch.from_numpy((rng.standard_normal((4, d)) * 0.02).astype(np.float32)).to(DEV).bfloat16()
    W[-4:] = last
    H = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(DEV).bfloat16()
    y = torch.tensor([V - 1, V - 3, -100], device=DEV)
    g = torch.ones(T, device=DEV)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    z = host(H) @ host(last).T
    want = np.log((V - 4) + np.exp(z).sum(axis=1))
    dz = d * 2.0 ** -23 * (np.abs(host(H)) @ np.abs(host(last)).T).max()
    assert (np.abs(host(lse) - want) <= 2 * dz + 2e-4).all()
    assert abs(float(loss[0]) - (want[0] - z[0, 3])) <= 2 * dz + 2e-4 and float(loss[2]) == 0
    p = np.exp(z - want[:, None])
    G = np.array([p[0] - np.eye(4)[3], p[1] - np.eye(4)[1]])
    ref = G.T @ host(H)[:2]
    assert np.abs(host(dW[-4:]) - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
    row = (np.exp(-want[:2])[:, None] * host(H)[:2]).sum(axis=0)
    assert np.abs(host(dW[123]) - row).max() <= 2.0 ** -6 * np.abs(row).max()
    refh = G @ host(last)
    assert np.abs(host(dH[:2]) - refh).max() <= 2.0 ** -7 * np.abs(refh).max() and not dH[2].any()


def test_no_tokens(q):
    H, W, y, g = make(4, 50, 16, "bf16", 3)
    dW = torch.full((50, 16), 7.0, dtype=torch.bfloat16, device=DEV)
    loss, lse = q.qamw_cross_entropy(H[:0], W, y[:0])
    dH, dW = q.qamw_cross_entropy_grad(H[:0], W, y[:0], lse, g[:0], dW=dW)
    torch.cuda.synchronize()
    assert loss.numel() == 0 and dH.shape == (0, 16) and not dW.any()


@pytest.mark.parametrize("T,dt", [(1, "bf16"), (150, "bf16"), (20, "f32")])
def test_other_stream_and_graph(q, T, dt):
    say(f"case stream and graph T={T} {dt}")
    V, d = 700, 64
    H, W, y, g = make(T, V, d, dt, 5)
    loss, lse = q.qamw_cross_entropy(H, W, y)
    dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    loss2, lse2 = q.qamw_cross_entropy(H, W, y, stream=side)
    dH2, dW2 = q.qamw_cross_entropy_grad(H, W, y, lse2, g, stream=side)
    side.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(dH, dH2) and torch.equal(dW, dW2)
    ws = torch.empty(max(q.qamw_cross_entropy_workspace_bytes(T, V, d, DT[dt]),
                         q.qamw_cross_entropy_grad_workspace_bytes(T, V, d, DT[dt])), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qamw_cross_entropy(H, W, y, loss=loss2, lse=lse2, workspace=ws)
        q.qamw_cross_entropy_grad(H, W, y, lse2, g, dH=dH2, dW=dW2, workspace=ws)
    for k in range(4):
        H.copy_(make(T, V, d, dt, 20 + k)[0])
        ws.fill_(255)
        for t in (loss2, lse2, dH2, dW2):
            t.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        loss, lse = q.qamw_cross_entropy(H, W, y)
        dH, dW = q.qamw_cross_entropy_grad(H, W, y, lse, g)
        torch.cuda.synchronize()
        assert torch.equal(loss, loss2) and torch.equal(dH, dH2) and torch.equal(dW, dW2)


def test_refusals(q):
    H, W, y, g = make(4, 20, 16, "f32", 1)
    _, lse = q.qamw_cross_entropy(H, W, y)
    for call in (lambda: q.qamw_cross_entropy(H.bfloat16(), W, y),
                 lambda: q.qamw_cross_entropy(H.half(), W.half(), y),
                 lambda: q.qamw_cross_entropy(H[:, :8], W, y),
                 lambda: q.qamw_cross_entropy(H, W, y.int()),
                 lambda: q.qamw_cross_entropy(H, W, y[:3]),
                 lambda: q.qamw_cross_entropy(H.cpu(), W, y),
                 lambda: q.qamw_cross_entropy_grad(H, W, y, lse, g.double()),
                 lambda: q.qamw_cross_entropy_grad(H, W, y, lse, g, dW=torch.empty(20, 8, device=DEV))):
        with pytest.raises(ValueError):
            call()
    from vector_codebook_codec_amd._lib import QamwError

    with pytest.raises(QamwError):                       # rows off 16-byte boundaries
        q.qamw_cross_entropy(H[:, 1:9], W[:, 1:9], y)
    with pytest.raises(QamwError):                       # d not a multiple of 8
        q.qamw_cross_entropy(H[:, :12], W[:, :12], y)
    with pytest.raises(QamwError):
        q.qamw_cross_entropy(H, W, y, workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
