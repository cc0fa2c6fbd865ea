"""GPU parity of the attention cache in 4 bits against the oracle
(oracle/mxfp4_cache.py); needs an MI355X.

Criteria:
  * write: codes and scales equal byte for byte, slots that are not written
    untouched; read: the same values bit for bit, rounded to nearest even
    where the type is narrower;
  * attention, element by element: |out - exact| <= u_out |exact| + e S with S
    = sum_t p_t |v_t| and e the relative error of the weights:
      - their rounding u_p, in the numerator alone: a bf16 number has 8
        significant bits, so one of them is off by up to half a step, 2^-8
        (bf16 alone), and each further one takes the rest down by as much
        again: 2^-16 where fp16 and 2^-24 where fp32 takes part;
      - the scores' error twice (numerator and sum): products of 4-bit values
        and of a query's 24 bits are exact, sums of d of them in fp32 are off by
        d 2^-24 of the products' magnitudes, here at most 48 after scaling;
        then one rounding of up to 40 before the exponential: (48 d + 40) 2^-24;
      - the exponential and the sums of L terms: (L + 8) 2^-24, twice;
    u_out is half a step of the output's type, and 2^-20 S covers the joining
    of wavefronts and shares; lse within the scores' error + (L + 8) 2^-24 +
    2^-24 |lse| + 1e-6;
  * over all elements, in the root mean square (it does not grow with L): 4e-3
    of the result's norm for bf16 out (two roundings of 1.7e-3 at most), 5e-4 for
    fp16 (2^-11 / sqrt(3) at most, 2.9e-4), 1e-5 for fp32.
"""
import sys

import numpy as np
import pytest

from oracle import mxfp4_cache as C

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TERMS = {"f32": 3, "f16": 2, "bf16": 1}
WEIGHT = {1: 2.0 ** -8, 2: 2.0 ** -16, 3: 2.0 ** -24}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
RMS = {1: 4e-3, 2: 5e-4, 3: 1e-5}


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


def heads_of(rng, T, heads, d, dt):
    gain = np.exp(0.7 * rng.standard_normal((heads, d)))
    return torch.from_numpy((rng.standard_normal((T, heads, d)) * gain).astype(np.float32)).to(DT[dt])


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("dt", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("T,heads,d,page", [(1, 1, 1, 16), (1, 32, 128, 16), (5, 3, 31, 16), (40, 2, 64, 32), (33, 5, 80, 16),
                                            (70, 1, 96, 64), (19, 8, 128, 16), (9, 2, 200, 16), (17, 3, 256, 128)])
def test_write_and_read(q, T, heads, d, page, dt):
    say(f"case write T={T} heads={heads} d={d} page={page} {dt}")
    rng = np.random.default_rng(T * 1000 + d)
    pages = T // page + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.15] = -1                           # padded tokens
    if T > 4:
        slots[1], slots[3] = pages * page, -(1 << 40)
    K, V = (heads_of(rng, T, heads, d, dt) for _ in (0, 1))
    codes, scales = q.qamw_mxfp4_cache_new(pages, heads, page, d)
    codes.fill_(0x5a), scales.fill_(0x7b)
    want_c, want_s = codes.cpu().numpy(), scales.cpu().numpy()
    s = torch.from_numpy(slots).to(DEV)
    q.qamw_mxfp4_cache_write(K.to(DEV), V.to(DEV), s, codes, scales)
    C.write(want_c, want_s, host(K), host(V), slots)
    torch.cuda.synchronize()
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    for out in ("f32", "bf16", "f16"):
        got = q.qamw_mxfp4_cache_read(codes, scales, s, d, out_dtype=DT[out])
        for a, b in zip(got, C.read(want_c, want_s, slots, d)):
            assert torch.equal(a.cpu(), torch.from_numpy(b).float().to(DT[out]))


# ------------------------------------------------------------------ attention
def make(q, seed, seqs, heads, d, page, spread=1.0, extra_cols=1):
    """A cache of quantised keys and values, filled by the package from seqs = [(queries, length)], pages in random
    order; slots past a sequence's end, and pages of nobody, hold NaN blocks."""
    rng = np.random.default_rng(seed)
    need = [-(-max(length, 0) // page) for _, length in seqs]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    cols = max(need) + extra_cols
    table = np.full((len(seqs), cols), -1, dtype=np.int32)
    slots, first = [], 0
    for b, (_, length) in enumerate(seqs):
        table[b, :need[b]] = order[first:first + need[b]]
        first += need[b]
        t = np.arange(length)
        slots.append(table[b, t // page].astype(np.int64) * page + t % page)
    slots = np.concatenate(slots)
    codes, scales = q.qamw_mxfp4_cache_new(pages, heads, page, d)
    codes.fill_(0x77), scales.fill_(255)
    K, V = (heads_of(rng, len(slots), heads, d, "f32").to(DEV) * spread for _ in (0, 1))
    q.qamw_mxfp4_cache_write(K, V, torch.from_numpy(slots).to(DEV), codes, scales)
    starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
    return rng, codes, scales, table, np.array([length for _, length in seqs], dtype=np.int32), starts


def check(got, lse, want, want_lse, S, dt, out, d, L, what=""):
    terms = max(TERMS[dt], TERMS[out])
    got, lse = host(got), host(lse)
    score = (48 * d + 40) * 2.0 ** -24
    e = WEIGHT[terms] + 2 * score + 2 * (L + 8) * 2.0 ** -24 + 2.0 ** -20
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
        bound = HALF_STEP[out] * np.abs(want) + e * S + (2.0 ** -25 if out == "f16" else 0)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    assert (off[~nan] <= bound[~nan]).all(), (what, (off[~nan] / np.maximum(bound[~nan], 1e-300)).max())
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    live = ~empty & ~np.isnan(want_lse)
    assert (np.abs(lse[live] - want_lse[live]) <= score + (L + 8) * 2.0 ** -24 + 2.0 ** -24 * np.abs(want_lse[live]) + 1e-6).all()
    if (~nan).any() and np.linalg.norm(want[~nan]) > 0:
        assert np.linalg.norm((got - want)[~nan]) <= max(RMS[terms], RMS[TERMS[out]]) * np.linalg.norm(want[~nan]), what


def attend(q, case, dt="bf16", out=None, causal=True, window=0, q_scale=1.0):
    seed, seqs, heads, group, d, page = case
    out = out or dt
    rng, codes, scales, table, lengths, starts = make(q, seed, seqs, heads, d, page)
    T = int(starts[-1])
    Q = torch.from_numpy((q_scale * rng.standard_normal((T, heads * group, d))).astype(np.float32)).to(DT[dt])
    dev = [torch.from_numpy(x).to(DEV) for x in (table, lengths, starts)]
    one = all(n == 1 for n, _ in seqs)
    got, lse = q.qamw_mxfp4_cache_attention(Q.to(DEV), codes, scales, dev[0], dev[1], starts=None if one else dev[2],
                                            max_queries=max(n for n, _ in seqs), causal=causal, window=window, out_dtype=DT[out])
    torch.cuda.synchronize()
    want = C.attention(host(Q), codes.cpu().numpy(), scales.cpu().numpy(), table, lengths, starts, float(np.float32(d ** -0.5)),
                       causal, window)
    check(got, lse, *want, dt, out, d, max(length for _, length in seqs), case)
    return got, lse


SINGLE = [
    (1, [(1, 1)], 1, 1, 1, 16), (2, [(1, 1), (1, 0), (1, 2)], 2, 1, 32, 16), (3, [(1, 17), (1, 33)], 1, 3, 31, 16),
    (4, [(1, 127), (1, 128), (1, 129)], 2, 4, 64, 32), (5, [(1, 300)], 5, 2, 80, 16), (6, [(1, 200), (1, 1)], 3, 16, 96, 64),
    (7, [(1, 1000)], 4, 1, 128, 16), (8, [(1, 260), (1, 515)], 8, 4, 128, 64), (9, [(1, 150)], 2, 17, 128, 128),
    (10, [(1, 333)], 2, 8, 160, 16), (11, [(1, 260)], 1, 40, 200, 32), (12, [(1, 700)], 2, 2, 256, 256),
    (13, [(1, 5000)], 1, 4, 128, 64),
]


@pytest.mark.parametrize("case", SINGLE, ids=[str(c[0]) for c in SINGLE])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_one_query(q, case, dt):
    say(f"case attend {case} {dt}")
    attend(q, case, dt)


CHUNKS = [
    (21, [(3, 3)], 1, 1, 32, 16), (22, [(2, 1), (5, 40), (1, 0), (0, 9)], 2, 2, 64, 16), (23, [(17, 130), (4, 300)], 2, 4, 128, 32),
    (24, [(100, 100), (33, 257)], 1, 3, 80, 16), (25, [(9, 600)], 2, 8, 128, 64), (26, [(65, 129), (1, 400)], 2, 1, 256, 16),
    (27, [(40, 50)], 1, 5, 96, 128), (28, [(130, 390)], 1, 2, 128, 16),
]


@pytest.mark.parametrize("case", CHUNKS, ids=[str(c[0]) for c in CHUNKS])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 37), (False, 50), (True, 1 << 40)])
def test_chunks(q, case, causal, window):
    say(f"case chunk {case} causal={causal} window={window}")
    attend(q, case, "bf16", causal=causal, window=window)


@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("f32", "bf16"), ("f16", "f32"), ("bf16", "f16"), ("f32", "f32"), ("f16", "f16")])
def test_chunk_types(q, dt, out):
    for case in CHUNKS[1:4] + CHUNKS[5:6]:
        say(f"case types {case} {dt} -> {out}")
        attend(q, case, dt, out, window=100)
