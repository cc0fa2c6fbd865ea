"""GPU tests of the attention cache at the limits of what its header allows:
more queries than a call names, blocks that the library never writes, weights
and scores beyond a type's ordinary range.  Needs an MI355X; criteria as in
test_gpu_cache.py where no other is stated.
"""
import numpy as np
import pytest

from oracle import mxfp4_cache as C
from test_gpu_cache import DEV, check, host, make, poisoned, q, say, simple  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def on_gpu(*arrays):
    return [torch.from_numpy(a).to(DEV) for a in arrays]


def exact(Q, codes, scales, table, lengths, starts, causal=True, window=0):
    back = lambda x: x if isinstance(x, np.ndarray) else x.cpu().numpy()  # noqa: E731
    return C.attention(host(Q), back(codes), back(scales), back(table), back(lengths), back(starts),
                       float(np.float32(Q.shape[2] ** -0.5)), causal, window)


@pytest.mark.parametrize("n", [1, 7, 300])
@pytest.mark.parametrize("length", [400, 6000])
def test_starts_of_any_value(q, n, length):
    """Entries at the ends of 32 bits: the sequences that lie inside are computed, of the buffers around out and lse no
    other row is written."""
    say(f"case starts n={n} length={length}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n, length=length)
    want = q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, n)
    low, high = -2 ** 31, 2 ** 31 - 1
    out, lse = torch.empty(3 * n + 8, *Q.shape[1:], dtype=Q.dtype, device=DEV), torch.empty(3 * n + 8, Q.shape[1], device=DEV)
    for entries, whole in (([0, n, low, low], 1), ([0, n, 2 * n, low], 2), ([0, n, n + low, low], 1), ([0, low, low + 5, low], 0),
                           ([high, low, low, low], 0), ([high, high, low, low], 0)):
        out.fill_(7.0), lse.fill_(9.0)
        wild = torch.tensor(entries, dtype=torch.int32, device=DEV)
        q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, wild, n, out=out[4:-4], lse=lse[4:-4])
        torch.cuda.synchronize()
        end = 4 + whole * n
        # [low, low + 5) and the like hold no query; [n, low) and [n + low, low) neither
        assert torch.equal(out[4:end], want[0][:whole * n]) and torch.equal(lse[4:end], want[1][:whole * n]), entries
        for rows in (slice(0, 4), slice(end, None)):
            assert (out[rows] == 7).all() and (lse[rows] == 9).all(), entries


# 16, 32 and 128 rows a workgroup, in one share of the tokens and in several; the last row asked for is inside a workgroup's
@pytest.mark.parametrize("n,most,group,d", [(40, 7, 4, 128), (60, 33, 4, 128), (300, 197, 4, 128), (30, 5, 5, 64), (12, 3, 3, 256)])
@pytest.mark.parametrize("length", [500, 6000])
def test_queries_past_max_queries_are_left(q, n, most, group, d, length):
    """Of a sequence with more than max_queries queries the first max_queries are computed, at their own places, and no
    other row is written."""
    say(f"case most n={n} most={most} group={group} d={d} length={length}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n, length=length, group=group, d=d, seqs=2)
    out, lse = torch.full_like(Q, 7.0), torch.full(Q.shape[:2], 9.0, device=DEV)
    q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, most, out=out, lse=lse)
    torch.cuda.synchronize()
    asked = torch.arange(2 * n) % n < most
    assert (out.cpu()[~asked] == 7).all() and (lse.cpu()[~asked] == 9).all()
    want = [x[asked.numpy()] for x in exact(Q, codes, scales, table, lengths, starts)]
    check(out.cpu()[asked], lse.cpu()[asked], *want, "bf16", "bf16", d, length)


@pytest.mark.parametrize("n", [1, 7, 300])
def test_starts_without_max_queries(q, n):
    """All of the sequences' queries are computed where the caller names no limit."""
    say(f"case no limit n={n}")
    Q, codes, scales, table, lengths, starts = simple(q, n=n, length=400)
    out, lse = torch.full_like(Q, 7.0), torch.full(Q.shape[:2], 9.0, device=DEV)
    q.qamw_mxfp4_cache_attention(Q, codes, scales, table, lengths, starts, out=out, lse=lse)
    torch.cuda.synchronize()
    check(out, lse, *exact(Q, codes, scales, table, lengths, starts), "bf16", "bf16", 128, 400)


@pytest.mark.parametrize("d,spread", [(128, 1.0), (128, 4.0), (96, 2.0), (72, 1.0)])
def test_lse_does_not_depend_on_how_many_queries(q, d, spread):
    """The same queries in a call of few rows a key head and in one of many.  Both sum exact products of bf16 queries and
    4-bit keys in fp32, so in the root mean square either's lse is as far from 64 bits as the other's: within twice, and
    half a step of fp32 at the result's size."""
    say(f"case lse d={d} spread={spread}")
    n, few, group, length, page = 300, 90, 4, 900, 32
    rng, codes, scales, table, lengths, starts = make(q, 91, [(n, length)], 2, d, page, spread=spread)
    Q = torch.from_numpy(rng.standard_normal((n, 2 * group, d)).astype(np.float32)).to(torch.bfloat16)
    want = exact(Q, codes, scales, table, lengths, starts)
    many = q.qamw_mxfp4_cache_attention(Q.to(DEV), codes, scales, *on_gpu(table, lengths, starts), n)
    late = q.qamw_mxfp4_cache_attention(Q[-few:].to(DEV), codes, scales, *on_gpu(table, lengths, np.array([0, few], dtype=np.int32)), few)
    torch.cuda.synchronize()
    rms = lambda x: float(np.sqrt(np.mean(np.square(x))))  # noqa: E731
    off_many, off_few = rms(host(many[1])[-few:] - want[1][-few:]), rms(host(late[1]) - want[1][-few:])
    say(f"  lse off by {off_many:.3g} in a call of many rows, {off_few:.3g} in one of few")
    assert off_many <= 2 * off_few + 2.0 ** -24 * rms(want[1][-few:])


@pytest.mark.parametrize("n", [4, 60, 200])
@pytest.mark.parametrize("score", [14.0, 16.0, 17.625])
def test_weights_far_below_the_largest(q, n, score):
    """Of every 128 tokens one, whose value is 0, has a score that far above the others': out is what they add up to.
    Their weights, exp(-score) of the largest, are 2^-20.2 to 2^-25.5 and round to within 2^-16 of themselves, or with
    many rows in bf16 to 2^-32 of the largest; then comes the output's half step.  The scores are exact, the sums of
    1024 terms within 1032 2^-24."""
    say(f"case weights n={n} score={score}")
    group, d, page, length = 4, 128, 64, 1024
    K, V = torch.zeros(length, 1, d), torch.ones(length, 1, d)
    K[::128, 0, 0], V[::128] = 1.0, 0.0
    table = torch.arange(length // page, dtype=torch.int32).view(1, -1)
    codes, scales = q.qamw_mxfp4_cache_new(length // page, 1, page, d)
    q.qamw_mxfp4_cache_write(K.to(DEV), V.to(DEV), torch.arange(length, device=DEV), codes, scales)
    Q = torch.zeros(n, group, d, dtype=torch.bfloat16)
    Q[:, :, 0] = score
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([length], [0, n])]
    got, lse = q.qamw_mxfp4_cache_attention(Q.to(DEV), codes, scales, table.to(DEV), dev[0], dev[1], n, scale=1.0, causal=False)
    torch.cuda.synchronize()
    weight = np.exp(-score)
    want = 127 * weight / (1 + 127 * weight)
    off = np.abs(host(got) / want - 1).max()
    assert off <= max(2.0 ** -16, 2.0 ** -32 / weight if n * group > 768 else 0) + 2.0 ** -8 + 2 * 1032 * 2.0 ** -24 + 1e-6, off
    assert np.abs(host(lse) - (score + np.log(8) + np.log1p(127 * weight))).max() <= 1032 * 2.0 ** -24 + 17 * 2.0 ** -23


LARGE = [  # queries, length, group, d: one query, a few rows, and (bf16) many rows
    (1, 700, 4, 128), (6, 260, 3, 80), (40, 400, 4, 128), (9, 200, 2, 256), (40, 300, 2, 64), (230, 600, 4, 128),
]


@pytest.mark.parametrize("dt,n,length,group,d", [("bf16", *c) for c in LARGE] + [("f32", *c) for c in LARGE[:-1]])
@pytest.mark.parametrize("code", [253, 254])
def test_values_past_every_number(q, n, length, group, d, code, dt):
    """Values with scale codes 253 and 254 stay with the rows that see their token: the other rows, and the other blocks of
    these, are as if the blocks were NaN, which the oracle gives to the same rows."""
    say(f"case code {code} n={n} length={length} group={group} d={d} {dt}")
    last = length - 1 if n == 1 else length - 2
    where = {0: [(1, last, 0, 0), (1, length - n // 2 - 1, 1, (d - 1) // 32), (1, 2, 0, 1)], 1: [(1, last, 1, 1)], 2: [(1, 5, 0, 0)]}
    rng, codes, scales, table, lengths, starts = poisoned(q, 79, [(n, length)] * 3, 2, d, 16, lambda b: where[b], code)
    Q = torch.from_numpy(rng.standard_normal((3 * n, 2 * group, d)).astype(np.float32)).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    nan = scales.cpu().numpy()
    nan[(nan == 253) | (nan == 254)] = 255
    for window in (0, max(1, n // 3)):
        got, lse = q.qamw_mxfp4_cache_attention(Q.to(DEV), codes, scales, *on_gpu(table, lengths, starts), n, window=window)
        torch.cuda.synchronize()
        with np.errstate(invalid="ignore"):
            want = exact(Q, codes, nan, table, lengths, starts, window=window)
            seen = torch.from_numpy(np.isnan(want[0]))
            check(got.cpu().masked_fill(seen, float("nan")), lse, *want, dt, dt, d, length)
            # a block's largest elements are infinite in fp32, in some of the rows that see them at least
            assert not torch.isfinite(got.cpu()[seen]).all(), (code, window)
