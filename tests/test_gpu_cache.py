"""GPU parity of the attention cache in 4 bits against the oracle
(oracle/mxfp4_cache.py); needs an MI355X.

Criteria:
  * write: codes and scales equal byte for byte, slots that are not written
    untouched; read: the same values bit for bit, rounded to nearest even
    where the type is narrower;
  * attention, element by element: |out - exact| <= u_out |exact| + e S with S
    = sum_t p_t |v_t| and e the relative error of the weights:
      - their rounding u_p, in the numerator alone: a bf16 number has 8
        significant bits, so one of them is off by up to half a step, 2^-8,
        and each further one takes the rest down by as much again: two for bf16
        and fp16, 2^-16, three where fp32 takes part, 2^-24; as fp16 (bf16 and
        many rows) half a step is 2^-11, or 2^-25 of the row's reference, which
        is at most the sum of its weights: up to 2^-25 sum_t |v_t| more;
      - the scores' error twice (numerator and sum): products of 4-bit values
        and of a query's 24 bits are exact, sums of d of them in fp32 are off by
        d 2^-24 of the products' magnitudes, here at most 48 after scaling;
        then one rounding of up to 40 before the exponential: (48 d + 40) 2^-24;
        bf16 and many rows (heads of 65 to 128): an instruction sums 128 products
        cut off below 24 bits of the largest, twice: 2 128 2^-24 48 = 48 2^-16;
      - the exponential and the sums of L terms: (L + 8) 2^-24, twice;
    u_out is half a step of the output's type, and 2^-20 S covers the joining
    of wavefronts and shares; lse within the scores' error + (L + 8) 2^-24 +
    2^-24 |lse| + 1e-6;
  * over all elements, in the root mean square (it does not grow with L): 2e-3
    of the result's norm for bf16 out (one rounding of 1.7e-3 at most), 5e-4 for
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
WEIGHT = {1: 2.0 ** -11, 2: 2.0 ** -16, 3: 2.0 ** -24}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
RMS = {1: 2e-3, 2: 5e-4, 3: 1e-5}


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


def check(got, lse, want, want_lse, S, plain, dt, out, d, L, what="", unit=1.0, mean=True):
    terms = max(TERMS[dt], TERMS[out])
    got, lse = host(got), host(lse)
    score = (48 * d + 40) * 2.0 ** -24 + (48 * 2.0 ** -16 if terms == 1 and 64 < d <= 128 else 0)
    e = WEIGHT[terms] + 2 * score + 2 * (L + 8) * 2.0 ** -24 + 2.0 ** -20
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
        bound = HALF_STEP[out] * np.abs(want) + e * S + (2.0 ** -25 if out == "f16" else 0)
        bound += 2.0 ** -25 * plain if terms == 1 else 0
    # products below fp32's normal numbers may count as 0: two numbers of the weight times L values, then the output's own
    tiny = (2 * L + 1) * 2.0 ** -126 / unit
    bound += tiny
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    assert (off[~nan] <= bound[~nan]).all(), (what, (off[~nan] / np.maximum(bound[~nan], 1e-300)).max())
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    live = ~empty & ~np.isnan(want_lse)
    assert (np.abs(lse[live] - want_lse[live]) <= score + (L + 8) * 2.0 ** -24 + 2.0 ** -24 * np.abs(want_lse[live]) + 1e-6).all()
    if (~nan).any() and np.linalg.norm(want[~nan]) > 0:
        # (where few mantissas make up the norm, half steps have no mean and only their bound is left)
        assert np.linalg.norm((got - want)[~nan]) <= max(0 if mean else HALF_STEP[out], RMS[terms], RMS[TERMS[out]]) * np.linalg.norm(want[~nan]) + tiny * got.size ** 0.5, what


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


# more than 768 rows a key head: the kernel of many rows (head sizes 65 to 128, bf16), beside the others at the same sizes
MANY = [
    (31, [(300, 300), (2, 700)], 1, 4, 128, 16), (32, [(130, 517), (129, 129), (0, 5), (1, 0)], 2, 8, 96, 64),
    (33, [(900, 1000)], 1, 1, 100, 128), (34, [(260, 1500)], 1, 4, 66, 256), (35, [(97, 2600)], 1, 8, 128, 32),
    (36, [(800, 310)], 1, 1, 64, 16), (37, [(400, 410)], 1, 2, 160, 32),
]


@pytest.mark.parametrize("case", MANY, ids=[str(c[0]) for c in MANY])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100), (False, 40)])
def test_many_rows(q, case, causal, window):
    say(f"case many rows {case} causal={causal} window={window}")
    attend(q, case, "bf16", causal=causal, window=window)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_many_rows_types(q, dt):
    say(f"case many rows {dt}")
    attend(q, MANY[1], dt, window=100)


def poisoned(q, seed, seqs, heads, d, page, slots_of, code=255):
    """A cache of make with the scale codes of some tokens' value or key blocks set: slots_of(b) -> [(kv, token, head, block)]."""
    rng, codes, scales, table, lengths, starts = make(q, seed, seqs, heads, d, page)
    s = scales.cpu().numpy()
    for b in range(len(seqs)):
        for kv, t, h, block in slots_of(b):
            s[kv, table[b, t // page], h, t % page, block] = code
    return rng, codes, torch.from_numpy(s).to(DEV), table, lengths, starts


POISON = [  # queries, length, group, d: one query, a few rows, many rows
    (1, 700, 4, 128), (1, 300, 2, 64), (6, 260, 3, 80), (40, 400, 4, 128), (80, 300, 4, 128), (230, 600, 4, 128), (9, 200, 2, 256),
]


@pytest.mark.parametrize("n,length,group,d", POISON)
def test_nan_blocks(q, n, length, group, d):
    """A NaN block of a value reaches the rows that see its token, in its 32 elements, and no other row; of a key every
    element of those rows."""
    say(f"case NaN blocks n={n} length={length} group={group} d={d}")
    where = {0: [(1, length - 3 if n > 3 else length - 1, 0, 0), (1, length - n // 2 - 1, 1, (d - 1) // 32), (1, 2, 0, 1)],
             1: [(0, length - 2 if n > 3 else 5, 1, 1)], 2: [(1, 5, 0, 0)]}
    seqs = [(n, length)] * 3
    rng, codes, scales, table, lengths, starts = poisoned(q, 77, seqs, 2, d, 16, lambda b: where[b])
    Q = torch.from_numpy(rng.standard_normal((3 * n, 2 * group, d)).astype(np.float32)).to(torch.bfloat16)
    dev = [torch.from_numpy(x).to(DEV) for x in (table, lengths, starts)]
    for window in (0, max(1, n // 3)):
        got, lse = q.qamw_mxfp4_cache_attention(Q.to(DEV), codes, scales, dev[0], dev[1], dev[2], n, window=window)
        torch.cuda.synchronize()
        want = C.attention(host(Q), codes.cpu().numpy(), scales.cpu().numpy(), table, lengths, starts, float(np.float32(d ** -0.5)),
                           True, window)
        with np.errstate(invalid="ignore"):
            check(got, lse, *want, "bf16", "bf16", d, length)


@pytest.mark.parametrize("n,length,group,d", POISON)
@pytest.mark.parametrize("code", [7, 100, 143, 200])
def test_values_of_any_scale(q, n, length, group, d, code):
    """Values beyond fp16's range, large and small ones, among others."""
    say(f"case values scaled by code {code} n={n} length={length} group={group} d={d}")
    seqs = [(n, length)]
    every = [(1, t, 1, b) for t in range(length) for b in range((d + 31) // 32)] if code < 127 else [(1, length // 2, 1, 1)]
    rng, codes, scales, table, lengths, starts = poisoned(q, 78, seqs, 2, d, 32, lambda b: every, code)
    Q = torch.from_numpy(rng.standard_normal((n, 2 * group, d)).astype(np.float32)).to(torch.bfloat16)
    dev = [torch.from_numpy(x).to(DEV) for x in (table, lengths, starts)]
    got, lse = q.qamw_mxfp4_cache_attention(Q.to(DEV), codes, scales, dev[0], dev[1], dev[2], n, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    want, want_lse, S, plain = C.attention(host(Q), codes.cpu().numpy(), scales.cpu().numpy(), table, lengths, starts,
                                           float(np.float32(d ** -0.5)))
    for heads in (slice(0, group), slice(group, 2 * group)):   # the norms of the two key heads differ by far
        unit = np.abs(want[:, heads]).max()
        check(got[:, heads].double() / unit, lse[:, heads], want[:, heads] / unit, want_lse[:, heads], S[:, heads] / unit,
              plain[:, heads] / unit, "bf16", "bf16", d, length, unit=unit, mean=code < 127)


@pytest.mark.parametrize("n,group", [(1, 4), (40, 4), (260, 4)])
def test_many_small_weights(q, n, group):
    """One token far above 8000 others, whose weights of about 2^-16 each make up an eighth of the sum."""
    say(f"case small weights n={n} group={group}")
    d, page, length = 128, 64, 8000
    K, V = torch.zeros(length, 1, d), torch.ones(length, 1, d)
    K[100, 0, 0], V[100] = 1.0, 0.0
    table = torch.arange(length // page, dtype=torch.int32).view(1, -1)
    codes, scales = q.qamw_mxfp4_cache_new(length // page, 1, page, d)
    q.qamw_mxfp4_cache_write(K.to(DEV), V.to(DEV), torch.arange(length, device=DEV), codes, scales)
    Q = torch.zeros(n, group, d, dtype=torch.bfloat16)
    Q[:, :, 0] = 11.0
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([length], [0, n])]
    got, lse = q.qamw_mxfp4_cache_attention(Q.to(DEV), codes, scales, table.to(DEV), dev[0], dev[1], n, scale=1.0)
    torch.cuda.synchronize()
    others = np.arange(length - n, length, dtype=np.float64) * np.exp(-11.0)
    want = others / (1 + others)
    # weights of 2^-15.9 have 9 bits in fp16 (2^-25 of 2^-16), all the same way off: 2^-9, and the output's half step
    assert (np.abs(host(got) - want[:, None, None]) <= (2.0 ** -9 + 2.0 ** -8) * want[:, None, None]).all()
    assert np.allclose(host(lse), (11.0 + np.log1p(others))[:, None], atol=1e-5)


# ------------------------------------------------------------------ layouts, pages, rows of nobody
def simple(q, seed=5, n=7, length=200, heads=2, group=3, d=128, page=32, dt="bf16", seqs=3):
    rng, codes, scales, table, lengths, starts = make(q, seed, [(n, length)] * seqs, heads, d, page)
    Q = torch.from_numpy(rng.standard_normal((n * seqs, heads * group, d)).astype(np.float32)).to(DT[dt]).to(DEV)
    return Q, codes, scales, torch.from_numpy(table).to(DEV), torch.from_numpy(lengths).to(DEV), torch.from_numpy(starts).to(DEV)


@pytest.mark.parametrize("n", [1, 7, 300])
def test_pages_outside_the_cache_are_masked(q, n):
    say(f"case bad pages n={n}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n, length=400)
    bad = table.clone()
    bad[0, 3], bad[1, 0], bad[1, 5], bad[2] = -1, codes.shape[1], 1 << 30, -5
    got, lse = q.qamw_mxfp4_cache_attention(Q, codes, scales, bad, lengths, starts, n, causal=False)
    torch.cuda.synchronize()
    want = C.attention(host(Q), codes.cpu().numpy(), scales.cpu().numpy(), bad.cpu().numpy(), lengths.tolist(), starts.tolist(),
                       float(np.float32(128 ** -0.5)), False)
    check(got, lse, *want, "bf16", "bf16", 128, 400)
    assert (got[2 * n:] == 0).all() and torch.isneginf(lse[2 * n:]).all()


@pytest.mark.parametrize("n", [1, 7, 300])
def test_lengths_outside_the_table(q, n):
    """A negative length counts as 0, one past the table's columns as those; an empty table leaves nothing."""
    say(f"case lengths n={n}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n, length=384)
    want = q.qamw_mxfp4_cache_attention(Q, codes, scales, table[:, :12].contiguous(), lengths, starts, n)
    far = torch.tensor([2 ** 31 - 1, -7, 384], dtype=torch.int32, device=DEV)
    got = q.qamw_mxfp4_cache_attention(Q, codes, scales, table[:, :12].contiguous(), far, starts, n)
    none = q.qamw_mxfp4_cache_attention(Q, codes, scales, table[:, :0], lengths, starts, n)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[:n], b[:n]) and torch.equal(a[2 * n:], b[2 * n:])
    assert (got[0][n:2 * n] == 0).all() and (none[0] == 0).all() and torch.isneginf(none[1]).all()


@pytest.mark.parametrize("n", [1, 7, 300])
def test_rows_of_no_sequence_stay(q, n):
    say(f"case rows of nobody n={n}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n)
    want = q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, n)
    more = torch.cat([Q[:2], Q, Q.repeat(2, 1, 1)[:5]])        # 5 rows behind, also where Q has 3
    out, lse = torch.full_like(more, 7.0), torch.full(more.shape[:2], 9.0, device=DEV)
    q.qamw_mxfp4_cache_attention(more, codes, scales, table, lengths, starts + 2, n, out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out[2:-5], want[0]) and torch.equal(lse[2:-5], want[1])
    for rows in (slice(0, 2), slice(-5, None)):
        assert (out[rows] == 7).all() and (lse[rows] == 9).all()
    # starts that leave the queries: rows inside are computed, nothing outside is touched
    wild = torch.tensor([0, n, 2 ** 31 - 1, -4], dtype=torch.int32, device=DEV)
    out.fill_(7.0)
    q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, wild, n, out=out[2:-5], lse=lse[2:-5])
    torch.cuda.synchronize()
    assert torch.equal(out[2:2 + n], want[0][:n]) and (out[:2] == 7).all() and (out[-5:] == 7).all()


@pytest.mark.parametrize("n,d", [(1, 128), (7, 80), (300, 128), (7, 33)])
def test_strides(q, n, d):
    """Queries and outputs as parts of wider tensors, by token and by head, at odd offsets; a table with a pitch."""
    say(f"case strides n={n} d={d}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n, d=d)
    want = q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, n)
    T, H, _ = Q.shape
    wide = torch.full((T, 3 * H * d + 1), float("nan"), dtype=Q.dtype, device=DEV)
    view = wide[:, 1:1 + H * d].view(T, H, d)
    view.copy_(Q)
    by_head = torch.full((H, T + 1, d + 3), 5.0, dtype=Q.dtype, device=DEV)
    out = by_head[:, :T, :d].transpose(0, 1)
    pitched = torch.full((table.shape[0], table.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
    pitched[:, :table.shape[1]] = table
    got, lse = q.qamw_mxfp4_cache_attention(view, codes, scales, pitched[:, :table.shape[1]], lengths, starts, n, out=out)
    torch.cuda.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(lse, want[1])
    assert (by_head[:, T] == 5).all() and (by_head[:, :, d:] == 5).all()


def test_write_strides_and_a_shared_head(q):
    """Keys and values as parts of one projection's output, and one head broadcast to all."""
    say("case write strides")
    rng = np.random.default_rng(3)
    T, heads, d, page = 37, 3, 100, 16
    qkv = torch.from_numpy(rng.standard_normal((T, 5 * heads * d + 1)).astype(np.float32)).to(torch.float16).to(DEV)
    K, V = qkv[:, 1:1 + heads * d].view(T, heads, d), qkv[:, 1 + heads * d:1 + 2 * heads * d].view(T, heads, d)[:, :1].expand(T, heads, d)
    slots = torch.arange(T, device=DEV).flip(0)
    codes, scales = q.qamw_mxfp4_cache_new(4, heads, page, d)
    q.qamw_mxfp4_cache_write(K, V, slots, codes, scales)
    K2 = torch.empty(heads, T, d + 5, dtype=torch.float16, device=DEV)[:, :, :d].transpose(0, 1)
    got = q.qamw_mxfp4_cache_read(codes, scales, slots, d, K=K2)
    torch.cuda.synchronize()
    want_c, want_s = C.new(4, heads, page, d)
    C.write(want_c, want_s, host(K), host(V), slots.tolist())
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales.cpu().numpy(), want_s)
    assert got[0] is K2
    for a, b in zip(got, C.read(want_c, want_s, slots.tolist(), d)):
        assert torch.equal(a.cpu().contiguous(), torch.from_numpy(b).to(torch.float16))


def test_empty_calls(q):
    say("case empty calls")
    Q, codes, scales, table, lengths, starts = simple(q, n=1)
    out, lse = q.qamw_mxfp4_cache_attention(Q[:0], codes, scales, table[:0], lengths[:0])
    assert out.shape == (0, 6, 128) and lse.shape == (0, 6)
    none_c, none_s = q.qamw_mxfp4_cache_new(0, 2, 32, 128)
    out, lse = q.qamw_mxfp4_cache_attention(Q, none_c, none_s, table, lengths)
    K, V = q.qamw_mxfp4_cache_read(none_c, none_s, torch.tensor([0, 5, -1], device=DEV), 128)
    q.qamw_mxfp4_cache_write(K, V, torch.tensor([0, 5, -1], device=DEV), none_c, none_s)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all() and (K == 0).all() and (V == 0).all()


def test_refusals(q):
    Q, codes, scales, table, lengths, starts = simple(q)
    ok = dict(Q=Q, codes=codes, scales=scales, table=table, lengths=lengths, starts=starts, max_queries=7)
    call = lambda **kw: q.qamw_mxfp4_cache_attention(**{**ok, **kw})  # noqa: E731
    for kw in (dict(Q=Q.cpu()), dict(Q=Q.double()), dict(Q=Q[:, :, :64]), dict(codes=codes[:, :-1]), dict(scales=scales[:1]),
               dict(table=table.long()), dict(table=table[0]), dict(lengths=lengths[:2]), dict(starts=starts[:3]),
               dict(lengths=lengths.long()), dict(lse=torch.empty(3, device=DEV)), dict(out=Q[:1]), dict(out_dtype=torch.float64),
               dict(table=table.t())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(window=-1),
               dict(max_queries=0), dict(starts=None), dict(Q=Q[:, :5]), dict(workspace=torch.empty(1, dtype=torch.uint8, device=DEV)[1:])):
        with pytest.raises((ValueError, RuntimeError)):
            if "workspace" in kw:
                big = simple(q, n=1, length=4000, seqs=1)
                q.qamw_mxfp4_cache_attention(*big[:5], **kw)
            else:
                call(**kw)


# ------------------------------------------------------------------ graphs and streams
def test_step_in_a_graph(q):
    """A serving step, write and attention, captured once and replayed with other inputs, eager work in between."""
    say("case graph")
    heads, group, d, page, B = 2, 4, 128, 16, 3
    codes, scales = q.qamw_mxfp4_cache_new(3 * 40 + 1, heads, page, d)
    other = tuple(t.clone() for t in (codes, scales))
    table = torch.randperm(3 * 40, device=DEV).to(torch.int32).view(B, 40)
    new = lambda *s: torch.randn(*s, device=DEV).to(torch.bfloat16)  # noqa: E731
    K, V, Q = new(B, heads, d), new(B, heads, d), new(B, heads * group, d)
    lengths, slots = torch.ones(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int64, device=DEV)

    def place(t):
        lengths.fill_(t + 1)
        slots.copy_(table[:, t // page].long() * page + t % page)

    def step(c):
        q.qamw_mxfp4_cache_write(K, V, slots, *c)
        return q.qamw_mxfp4_cache_attention(Q, *c, table, lengths)

    place(0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step((codes, scales))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = step((codes, scales))
    for t in (0, 1, 15, 16, 200, 17, 600):
        place(t)
        for x in (K, V, Q):
            x.copy_(new(*x.shape))
        want = step(other)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(codes, other[0]) and torch.equal(scales, other[1])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), t


@pytest.mark.parametrize("n", [1, 300])
def test_on_another_stream(q, n):
    """Results and workspaces of a call on a stream that is not the current one, busy with other work."""
    say(f"case stream n={n}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n, length=3000, seqs=1)
    want = [x.clone() for x in q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, n)]
    a = torch.ones(4096, 4096, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a @ a
    got = q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, n, stream=side)
    again = q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, n, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for r in (got, again):
        assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


@pytest.mark.parametrize("n", [1, 300])
def test_offsets_past_32_bits(q, n):
    """Pages more than 4 GiB from the start of either half of the cache."""
    say(f"case large cache n={n}")
    heads, d, page, length = 8, 128, 64, 500
    Q, codes, scales, table, lengths, starts = simple(q, n=n, length=length, heads=heads, group=4, d=d, page=page, seqs=1)
    want = q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, n)
    t = torch.arange(length, device=DEV)
    old = table[0, t // page].long() * page + t % page
    pages = 140000
    far = torch.tensor([pages - 1 - 17 * i if i % 2 else 3 * i for i in range(table.shape[1])], dtype=torch.int32, device=DEV).view(1, -1)
    K, V = q.qamw_mxfp4_cache_read(codes, scales, old, d)
    big = q.qamw_mxfp4_cache_new(pages, heads, page, d)
    new = far[0, t // page].long() * page + t % page
    q.qamw_mxfp4_cache_write(K, V, new, *big)
    again = q.qamw_mxfp4_cache_read(*big, new, d)
    got = q.qamw_mxfp4_cache_attention(Q, *big, far, lengths, starts, n)
    torch.cuda.synchronize()
    assert torch.equal(again[0], K) and torch.equal(again[1], V)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
