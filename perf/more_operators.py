"""The 4-bit attention cache and the adapters beside the 4-bit product: the cases they are measured on.

A case names one operator and its sizes:

  store    keys and values of T tokens quantised into the cache's slots, and read back from there
  read     keys and values of T tokens read back from the cache
  attend   attention of B sequences over the cache: one query each, or a chunk of each one's latest tokens
  adapt    Y = Q(X) W_hat^T + f_i (X A_i^T) B_i^T, with an adapter i of its own for every request

The cache holds blocks of 32 elements of a head in 4 bits with one power-of-two scale each: codes
[2][pages][heads][page][16 ceil(d / 32)] and scales [2][pages][heads][page][2, 4 or 8], keys first.

``run`` computes them in plain torch operations in fp32 (``own`` false) or by the package's entry points
(``own`` true); ``exact`` in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_DEV = "cuda"
BLOCK = 32


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a single new token of one layer, 32 key and value heads: latency
        dict(name="store_1x32x128", op="store", T=1, heads=32, d=128, page=16, dtype="bf16"),
        # a prompt of odd length of one layer with grouped heads
        dict(name="store_8191x8x128", op="store", T=8191, heads=8, d=128, page=64, dtype="bf16"),
        # a short prefix of an odd head size back in fp32, as a check of the cache's error takes it
        dict(name="read_300x5x80_f32", op="read", T=300, heads=5, d=80, page=16, dtype="f32"),
        # the cached prefixes of a batch handed to another stage in bf16
        dict(name="read_65536x8x128", op="read", T=65536, heads=8, d=128, page=64, dtype="bf16"),
        # the next token of one short dialogue, as many key heads as query heads
        dict(name="attend_1x1000_32_32", op="attend", B=1, n=1, L=1000, q_heads=32, heads=32, d=128, page=16, dtype="bf16",
             causal=True, window=0),
        # the next token of each of 64 sequences of uneven length
        dict(name="attend_64x8192_32_8", op="attend", B=64, n=1, L=8192, q_heads=32, heads=8, d=128, page=64, dtype="bf16",
             causal=True, window=0),
        # a few long documents under a wide model
        dict(name="attend_4x131072_64_8", op="attend", B=4, n=1, L=131072, q_heads=64, heads=8, d=128, page=64, dtype="bf16",
             causal=True, window=0),
        # the latest pieces of four prompts, each behind what the cache holds of it
        dict(name="attend_4x2048_of_8192_32_8", op="attend", B=4, n=2048, L=8192, q_heads=32, heads=8, d=128, page=64,
             dtype="bf16", causal=True, window=0),
        # a few tokens a sequence to be verified at once, small heads, a sliding window, fp16
        dict(name="attend_8x5_of_3001_f16_window", op="attend", B=8, n=5, L=3001, q_heads=12, heads=4, d=64, page=32, dtype="f16",
             causal=True, window=1024),
        # one token through a gate projection with its request's adapter
        dict(name="adapt_1_11008x4096_r16", op="adapt", T=1, R=1, n=1, r=16, N=11008, d=4096, dtype="bf16", out="bf16"),
        # a decode batch of 48 requests with adapters of their own
        dict(name="adapt_48_4096x4096_r16", op="adapt", T=48, R=48, n=48, r=16, N=4096, d=4096, dtype="bf16", out="bf16"),
        # prompts of eight requests of odd lengths through a 13B-shaped projection, some of them with the same adapter
        dict(name="adapt_4095_13824x5120_r64", op="adapt", T=4095, R=8, n=3, r=64, N=13824, d=5120, dtype="bf16", out="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend", "attend", "adapt", "adapt"])
    if op == "adapt":
        T = _spread(rng, 1, 8192)
        R = min(T, _spread(rng, 1, 64))
        c = dict(op=op, T=T, R=R, n=rng.randint(1, R), r=_spread(rng, 1, 128), N=_spread(rng, 1, 13824),
                 d=_spread(rng, 1, 13824), dtype=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
        while c["T"] * c["N"] * c["d"] > 4095 * 13824 * 5120:
            c["N"], c["d"] = (c["N"] + 1) // 2, (c["d"] + 1) // 2
        return c
    heads, d, page = rng.choice([1, 2, 4, 5, 8, 32]), rng.choice([32, 64, 80, 96, 128, 128, 192, 256]), 16 << rng.randint(0, 4)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op != "attend":
        return dict(op=op, T=_spread(rng, 1, min(65536, (1 << 26) // (heads * d))), heads=heads, d=d, page=page, dtype=dtype)
    B, L = _spread(rng, 1, 64), _spread(rng, 1, 131072)
    while B * L * heads * d > 1 << 29:
        B, L = (B + 1) // 2, max(1, L * 3 // 4)
    n = 1 if rng.random() < 0.5 else _spread(rng, 1, min(L, 2048))
    group = rng.choice([1, 2, 3, 4, 8])
    most = (1 << 38) // (64 if dtype == "f32" else 4)            # rows x tokens x d
    while B * n * heads * group * L * d > most and n > 1:
        n = max(1, n * 3 // 4)
    return dict(op=op, B=B, n=n, L=L, q_heads=heads * group, heads=heads, d=d, page=page, dtype=dtype,
                causal=rng.random() < 0.8, window=rng.choice([0, 0, _spread(rng, 1, L)]))


# ------------------------------------------------------------------ what a case's sequences and requests are
def _sequences(c):
    """(queries, cached tokens) of each sequence: uneven, the first one the longest; the queries are the latest tokens."""
    out = []
    for j in range(c["B"]):
        n = max(1, c["n"] - (j * 37) % (c["n"] // 2 + 1))
        out.append((n, max(n, c["L"] - (j * 7919) % (c["L"] // 2 + 1))))
    return out


def _spans(c):
    """Of each sequence: the first cached token that any query attends to, and the pairs of query and token."""
    out = []
    for n, length in _sequences(c):
        first, pairs = length, 0
        for i in range(n):
            hi = length - n + i + 1 if c["causal"] else length
            lo = max(0, length - n + i + 1 - c["window"]) if c["window"] else 0
            first, pairs = min(first, lo), pairs + hi - lo
        out.append((first, pairs))
    return out


def _requests(c):
    """(tokens, adapter) of each request, the tokens in order; every fifth request goes without an adapter."""
    T, R = c["T"], c["R"]
    cuts = [T * j // R for j in range(R + 1)]
    for j in range(1, R):                                        # odd lengths
        if cuts[j - 1] < cuts[j] - 1:
            cuts[j] -= cuts[j] & 1 ^ 1
    return [(cuts[j + 1] - cuts[j], -1 if j % 5 == 4 else j % c["n"]) for j in range(R)]


# ------------------------------------------------------------------ inputs
def _heads(g, T, heads, d, dtype):
    """Keys or values of T tokens: a few channels of each head are several times larger, as trained ones are."""
    gain = torch.exp(0.7 * torch.randn(heads, d, device=_DEV, generator=g))
    return (torch.randn(T, heads, d, device=_DEV, generator=g) * gain).to(dtype)


def _new_cache(pages, heads, page, d):
    nb = (d + BLOCK - 1) // BLOCK
    sb = 2 if nb <= 2 else 4 if nb <= 4 else 8
    return (torch.zeros(2, pages, heads, page, 16 * nb, dtype=torch.uint8, device=_DEV),
            torch.zeros(2, pages, heads, page, sb, dtype=torch.uint8, device=_DEV))


def _fill(g, codes, scales, slots, d):
    """Quantised keys and values of another generator into the given slots, some tokens at a time."""
    heads, page = codes.shape[2], codes.shape[3]
    step = max(1, (1 << 25) // (heads * d))
    for i in range(0, slots.numel(), step):
        at = slots[i:i + step]
        for kv in (0, 1):
            c, s = _pack(_heads(g, at.numel(), heads, d, torch.bfloat16))
            codes[kv, at // page, :, at % page] = c
            scales[kv, at // page, :, at % page] = torch.nn.functional.pad(s, (0, scales.shape[4] - s.shape[2]))


def _weights(g, rows, cols, dtype, std=0.02):
    w = torch.randn(rows, cols, device=_DEV, generator=g)
    w *= torch.exp(0.3 * torch.randn(rows, cols, device=_DEV, generator=g))
    return w.mul_(std / 1.09).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    op, d = case["op"], case["d"]
    s = {"case": case}
    if op == "adapt":
        T, N, r, n, dtype = case["T"], case["N"], case["r"], case["n"], _DT[case["dtype"]]
        gain = torch.exp(0.5 * torch.randn(d, device=_DEV, generator=g))
        s["X"] = (torch.randn(T, d, device=_DEV, generator=g) * gain).to(dtype)
        s["codes"], s["scales"] = _pack(_weights(g, N, d, torch.float32))
        s["scales"] = torch.nn.functional.pad(s["scales"], (0, -s["scales"].shape[1] % 16)).contiguous()
        s["A"] = _weights(g, n * r, d, dtype, d ** -0.5).view(n, r, d)
        s["B"] = _weights(g, n * N, r, dtype, 0.02).view(n, N, r)
        s["factors"] = torch.rand(n, device=_DEV, generator=g) + 0.5
        s["index"] = torch.cat([torch.full((t,), i, dtype=torch.int32) for t, i in _requests(case)]).to(_DEV)
        return s
    heads, page = case["heads"], case["page"]
    if op in ("store", "read"):
        T = case["T"]
        pages = (T + page - 1) // page + 3
        s["codes"], s["scales"] = _new_cache(pages, heads, page, d)
        order = torch.randperm(pages, device=_DEV, generator=g)
        t = torch.arange(T, device=_DEV)
        s["slots"] = order[t // page] * page + t % page
        if op == "read":
            _fill(g, s["codes"], s["scales"], s["slots"], d)
        else:
            s["K"], s["V"] = (_heads(g, T, heads, d, _DT[case["dtype"]]) for _ in (0, 1))
        return s
    seq = _sequences(case)
    need = [(length + page - 1) // page for _, length in seq]
    pages = sum(need) + 3
    s["codes"], s["scales"] = _new_cache(pages, heads, page, d)
    order = torch.randperm(pages, device=_DEV, generator=g).to(torch.int32)
    table = torch.full((case["B"], max(need) + 2), -1, dtype=torch.int32, device=_DEV)
    first = 0
    for b, (n, length) in enumerate(seq):
        table[b, :need[b]] = order[first:first + need[b]]
        first += need[b]
        t = torch.arange(length, device=_DEV)
        _fill(g, s["codes"], s["scales"], table[b, t // page].long() * page + t % page, d)
    s["table"] = table
    s["lengths"] = torch.tensor([length for _, length in seq], dtype=torch.int32, device=_DEV)
    starts = [0]
    for n, _ in seq:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=_DEV)
    s["Q"] = (1.5 * torch.randn(starts[-1], case["q_heads"], d, device=_DEV, generator=g)).to(_DT[case["dtype"]])
    return s


# ------------------------------------------------------------------ plain forms (fp32)
_MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise_plain(v):
    """(element index 0..7, negative?, scale code) of the blocks along the last axis."""
    v = v.float()
    v = torch.nn.functional.pad(v, (0, -v.shape[-1] % BLOCK))
    b = v.view(*v.shape[:-1], -1, BLOCK)
    m = b.abs().amax(dim=-1)
    e = torch.frexp(m)[1] - 3                                   # floor(log2 m) - 2
    e = torch.where(m > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    idx = torch.zeros(a.shape, dtype=torch.uint8, device=a.device)
    # edges between neighbouring elements; a tie goes to the even index
    for edge, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        idx += (a >= edge) if tie_up else (a > edge)
    return idx, torch.signbit(b), (e + 127).to(torch.uint8)


def _values_plain(idx, neg, code, d):
    mag = torch.tensor(_MAG, device=idx.device)[idx.int()]
    val = torch.ldexp(torch.where(neg, -mag, mag), code.int().unsqueeze(-1) - 127)
    return val.flatten(-2)[..., :d]


def _pack(v):
    """Codes (low nibble first) and one scale code per block."""
    idx, neg, code = _quantise_plain(v)
    nib = (idx | (neg.to(torch.uint8) << 3)).flatten(-2)
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).contiguous(), code.contiguous()


def _unpack_plain(codes, scales, d):
    nib = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    nib = nib.view(*nib.shape[:-1], -1, BLOCK)
    return _values_plain(nib & 7, nib >= 8, scales[..., :nib.shape[-2]], d)


def _read_plain(codes, scales, slots, d):
    page = codes.shape[3]
    return [_unpack_plain(codes[kv, slots // page, :, slots % page], scales[kv, slots // page, :, slots % page], d)
            for kv in (0, 1)]


def _allowed(n, length, causal, window, device):
    """[n][length]: which cached tokens a query attends to."""
    at = torch.arange(length - n, length, device=device).unsqueeze(1)
    t = torch.arange(length, device=device).unsqueeze(0)
    ok = (t <= at) if causal else torch.ones(n, length, dtype=torch.bool, device=device)
    return ok & (t > at - window) if window else ok


def _attend_plain(s):
    c = s["case"]
    d, heads, group, page = c["d"], c["heads"], c["q_heads"] // c["heads"], c["page"]
    out = torch.empty(s["Q"].shape, dtype=s["Q"].dtype, device=s["Q"].device)
    lse = torch.empty(s["Q"].shape[:2], device=s["Q"].device)
    first = 0
    for b, (n, length) in enumerate(_sequences(c)):
        t = torch.arange(length, device=out.device)
        k, v = _read_plain(s["codes"], s["scales"], s["table"][b, t // page].long() * page + t % page, d)
        q = s["Q"][first:first + n].float().view(n, heads, group, d).permute(1, 2, 0, 3).reshape(heads, group * n, d)
        z = torch.matmul(q, k.permute(1, 2, 0).contiguous()).mul_(d ** -0.5)
        z = z.view(heads, group, n, length).masked_fill_(~_allowed(n, length, c["causal"], c["window"], out.device), float("-inf"))
        m = z.amax(dim=-1, keepdim=True)
        p = torch.exp(z.sub_(m))
        total = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.div_(total).view(heads, group * n, length), v.permute(1, 0, 2).contiguous())
        out[first:first + n] = o.view(heads, group, n, d).permute(2, 0, 1, 3).reshape(n, heads * group, d).to(out.dtype)
        lse[first:first + n] = (m + torch.log(total)).squeeze(-1).permute(2, 0, 1).reshape(n, heads * group)
        first += n
    return out, lse


def _adapt_plain(s):
    c = s["case"]
    d = c["d"]
    X = s["X"].float()
    y = torch.matmul(_values_plain(*_quantise_plain(s["X"]), d), _unpack_plain(s["codes"], s["scales"], d).t())
    first = 0
    for tokens, i in _requests(c):
        if i >= 0:
            u = torch.matmul(X[first:first + tokens], s["A"][i].float().t()) * s["factors"][i]
            y[first:first + tokens] += torch.matmul(u, s["B"][i].float().t())
        first += tokens
    return y.to(_DT[c["out"]])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "store":
        page = c["page"]
        for kv, x in enumerate((s["K"], s["V"])):
            codes, scales = _pack(x)
            s["codes"][kv, s["slots"] // page, :, s["slots"] % page] = codes
            s["scales"][kv, s["slots"] // page, :, s["slots"] % page] = torch.nn.functional.pad(
                scales, (0, s["scales"].shape[4] - scales.shape[2]))
    if c["op"] in ("store", "read"):
        return tuple(x.to(_DT[c["dtype"]]) for x in _read_plain(s["codes"], s["scales"], s["slots"], c["d"]))
    return _attend_plain(s) if c["op"] == "attend" else _adapt_plain(s)


# ------------------------------------------------------------------ the package's entry points
def _run_own(s):
    import vector_codebook_codec_amd as q

    c = s["case"]
    if c["op"] == "adapt":
        return q.qamw_mxfp4_adapter_matmul(s["X"], s["codes"], s["scales"], s["A"], s["B"], s["index"], s["factors"],
                                           out_dtype=_DT[c["out"]])
    if c["op"] == "attend":
        return q.qamw_mxfp4_cache_attention(s["Q"], s["codes"], s["scales"], s["table"], s["lengths"],
                                            starts=None if c["n"] == 1 else s["starts"], max_queries=c["n"],
                                            causal=c["causal"], window=c["window"])
    if c["op"] == "store":
        q.qamw_mxfp4_cache_write(s["K"], s["V"], s["slots"], s["codes"], s["scales"])
    return q.qamw_mxfp4_cache_read(s["codes"], s["scales"], s["slots"], c["d"], out_dtype=_DT[c["dtype"]])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, d = case["op"], case["d"]
    nb = (d + BLOCK - 1) // BLOCK
    size = _SIZE[case["dtype"]]
    if op in ("store", "read"):
        rows = 2 * case["T"] * case["heads"]
        moved = rows * (d * size + 17 * nb)                      # one side in 4 bits, the other in dtype
        return {"bytes": (2 if op == "store" else 1) * moved + 8 * case["T"], "flops": rows * d}
    if op == "attend":
        seq, spans = _sequences(case), _spans(case)
        tokens = sum(length - first for (_, length), (first, _) in zip(seq, spans))
        queries = sum(n for n, _ in seq)
        return {"bytes": tokens * case["heads"] * 2 * 17 * nb + queries * case["q_heads"] * (2 * d * size + 4),
                "flops": 4 * d * case["q_heads"] * sum(pairs for _, pairs in spans)}
    T, N, r = case["T"], case["N"], case["r"]
    req = _requests(case)
    used, with_one = len({i for _, i in req if i >= 0}), sum(t for t, i in req if i >= 0)
    return {"bytes": T * d * size + 17 * N * nb + used * r * (d + N) * size + 4 * T + T * N * _SIZE[case["out"]],
            "flops": 2 * T * N * d + 2 * with_one * r * (d + N)}


# ------------------------------------------------------------------ 64-bit definition
def _mx64(v):
    """Nearest element by distance to each of the eight, ties to the even one: the values, float64."""
    v = v.double()
    d = v.shape[-1]
    nb = (d + BLOCK - 1) // BLOCK
    full = torch.zeros(*v.shape[:-1], nb * BLOCK, dtype=torch.float64, device=v.device)
    full[..., :d] = v
    full = full.view(*v.shape[:-1], nb, BLOCK)
    m = full.abs().max(dim=-1).values
    e = torch.floor(torch.log2(torch.where(m > 0, m, torch.ones_like(m))))
    e = e - (torch.exp2(e) > m).double() + (torch.exp2(e + 1) <= m).double()
    scale = torch.exp2(torch.where(m > 0, e - 2, torch.full_like(m, -127.0)).clamp(-127, 127)).unsqueeze(-1)
    best, mag, a = torch.full_like(full, float("inf")), torch.zeros_like(full), full.abs() / scale
    for i in (0, 2, 4, 6, 1, 3, 5, 7):                          # even elements first, so that they keep their ties
        dist = (a - _MAG[i]).abs()
        closer = dist < best
        mag = torch.where(closer, torch.full_like(mag, _MAG[i]), mag)
        best = torch.where(closer, dist, best)
    return (torch.copysign(mag, full) * scale).reshape(*v.shape[:-1], nb * BLOCK)[..., :d]


def _decode64(codes, scales, d):
    sixteen = torch.tensor(_MAG + tuple(-m for m in _MAG), dtype=torch.float64, device=codes.device)
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    out[..., 0::2] = sixteen[(codes % 16).long()]
    out[..., 1::2] = sixteen[(codes // 16).long()]
    nb = out.shape[-1] // BLOCK
    return (out * torch.exp2(scales[..., :nb].double() - 127.0).repeat_interleave(BLOCK, dim=-1))[..., :d]


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "store":
        return _mx64(s["K"]), _mx64(s["V"])
    if case["op"] == "read":
        page = case["page"]
        rows = [x.transpose(2, 3).flatten(1, 2) for x in (s["codes"], s["scales"])]      # [2][slots][heads][...]
        out = torch.empty(2, case["T"], case["heads"], d, dtype=torch.float64, device=_DEV)
        for i in range(0, case["T"], 4096):
            at = s["slots"][i:i + 4096]
            for kv in (0, 1):
                out[kv, i:i + 4096] = _decode64(rows[0][kv, at], rows[1][kv, at], d)
        return out[0], out[1]
    if case["op"] == "adapt":
        Y = torch.matmul(_mx64(s["X"]), _decode64(s["codes"], s["scales"], d).t())
        X = s["X"].double()
        for i in range(case["n"]):
            rows = (s["index"] == i).nonzero().squeeze(1)
            if rows.numel():
                low = torch.matmul(X[rows], s["A"][i].double().t())
                Y[rows] += float(s["factors"][i]) * torch.matmul(low, s["B"][i].double().t())
        return Y
    # head by head and sequence by sequence, the queries in pieces
    group, page = case["q_heads"] // case["heads"], case["page"]
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.zeros(s["Q"].shape[:2], dtype=torch.float64, device=_DEV)
    starts = s["starts"].tolist()
    for b, length in enumerate(s["lengths"].tolist()):
        used = s["table"][b, :(length + page - 1) // page].long()
        n = starts[b + 1] - starts[b]
        for h in range(case["heads"]):
            k, v = (_decode64(s["codes"][kv, used, h], s["scales"][kv, used, h], d).flatten(0, 1)[:length] for kv in (0, 1))
            kt = k.t().contiguous()
            for i in range(0, n, 512):
                rows = slice(starts[b] + i, starts[b] + min(i + 512, n))
                own_place = length - n + torch.arange(i, min(i + 512, n), device=_DEV)
                gap = own_place.unsqueeze(1) - torch.arange(length, device=_DEV)         # tokens back from the query's own
                hidden = torch.zeros_like(gap, dtype=torch.bool)
                if case["causal"]:
                    hidden |= gap < 0
                if case["window"]:
                    hidden |= gap >= case["window"]
                for j in range(h * group, (h + 1) * group):
                    z = torch.mm(s["Q"][rows, j].double(), kt) / math.sqrt(d)
                    z = torch.where(hidden, torch.full_like(z, float("-inf")), z)
                    lse[rows, j] = torch.logsumexp(z, dim=1)
                    out[rows, j] = torch.mm(torch.exp(z - lse[rows, j].unsqueeze(1)), v)
    return out, lse
