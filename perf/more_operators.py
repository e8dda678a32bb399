"""Cases of a key-value cache held in 4 bits, and of what stands in the same pass as the
write into a cache: norms of each head's queries and keys, and positions of several axes.

attention   softmax attention of the new tokens' queries over a paged cache of 4-bit
            codes, each 32 values of a token's head with a scale of their own.
kv_append   norms of queries and keys (optional), rotary positions of one or several axes
            (optional), and the write into the 4-bit cache, or into the 8-bit one.

`run` computes them with elementary torch operations, or, where `own` is true, calls
the library's operators.
"""
import math
import random

import torch

own = False

GROUP = 32                            # values that share a scale (4 bits)
SCALE_MIN, SCALE_MAX = 2.0 ** -14, 57344.0     # limits of a scale: e5m2 numbers
EXP_MIN, EXP_MAX = -64, 64            # limits of a page's exponent (8 bits)
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One user, short prompt: latency is all there is (heads of an 8B decoder).
        dict(name="attn4-decode-1", op="attention", batch=1, new=1, len=257, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # One user at the end of a long document: the cache is read once.
        dict(name="attn4-decode-long", op="attention", batch=1, new=1, len=131001, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # A serving batch whose sequences have very different lengths.
        dict(name="attn4-decode-batch", op="attention", batch=64, new=1, len=16001, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # Heads of a 1B decoder, small pages, a sliding window that cuts most pages off.
        dict(name="attn4-decode-window", op="attention", batch=96, new=1, len=3001, ragged=True,
             heads=32, kv_heads=8, dim=64, page=16, window=1000),
        # Checking five guessed tokens a sequence at once, seven heads per key-value head.
        dict(name="attn4-verify", op="attention", batch=8, new=5, len=6001, ragged=True,
             heads=28, kv_heads=4, dim=128, page=64, window=0),
        # A whole prompt.
        dict(name="attn4-prefill", op="attention", batch=1, new=4096, len=4096, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # Chunks of several prompts behind what is cached of them already.
        dict(name="attn4-chunk", op="attention", batch=4, new=701, len=9001, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # A decode step of one user of a decoder with head norms: one token.
        dict(name="append4-decode-1", op="kv_append", bits=4, batch=1, new=1, len=300, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, rotary=128, interleaved=False, norm=True, axes=0),
        # Prompts of such a decoder.
        dict(name="append4-prefill", op="kv_append", bits=4, batch=2, new=8001, len=8001, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, rotary=128, interleaved=False, norm=True, axes=0),
        # Text with an image in it: positions of time, height and width, no norms.
        dict(name="append4-image", op="kv_append", bits=4, batch=1, new=5003, len=5003, ragged=False,
             heads=28, kv_heads=4, dim=128, page=64, rotary=128, interleaved=False, norm=False, axes=3),
        # A decode batch into the 8-bit cache, with head norms and three axes.
        dict(name="append8-decode-batch", op="kv_append", bits=8, batch=64, new=1, len=1000, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, rotary=128, interleaved=False, norm=True, axes=3),
        # Prompts into the 8-bit cache with head norms.
        dict(name="append8-prefill", op="kv_append", bits=8, batch=2, new=8001, len=8001, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, rotary=128, interleaved=False, norm=True, axes=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "kv_append", "kv_append"])
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (32, 8), (16, 16), (40, 8), (16, 2), (16, 1)])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    if op == "kv_append":
        batch = _log(rng, 1, 64)
        new = rng.choice([1, _log(rng, 1, 16002 // batch)])
        bits, norm, axes = rng.choice([4, 4, 8]), rng.random() < 0.6, rng.choice([0, 0, 1, 2, 3])
        return dict(op=op, bits=bits, batch=batch, new=new, len=new + _log(rng, 1, 4000 // batch + 1) - 1,
                    ragged=rng.random() < 0.5, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    rotary=rng.choice([dim, dim, dim // 2, dim // 4 * 3, 10]), interleaved=rng.random() < 0.4,
                    norm=norm or (bits == 8 and axes == 0), axes=axes)
    kind = rng.choice(["decode", "decode", "verify", "prefill"])
    if kind == "prefill":
        batch = _log(rng, 1, 6)
        new = _log(rng, 17, 4096 // batch)
        length = new + rng.choice([0, _log(rng, 1, 12000 // batch)])
        length = min(length, 8 * 1024 * 1024 * 32 // (heads * batch * new))
        length = max(length, new)
    else:
        batch = _log(rng, 1, 96)
        new = 1 if kind == "decode" else rng.randint(2, 16)
        length = max(new, _log(rng, 1, 131001 // batch))
    return dict(op=op, batch=batch, new=new, len=length, ragged=rng.random() < 0.6, heads=heads, kv_heads=kv_heads,
                dim=dim, page=page, window=rng.choice([0, 0, 0, _log(rng, 1, 4000)]))


def _lengths(case):
    """(lengths after the call, new tokens) of each sequence: of the case alone."""
    rng = random.Random("%(batch)d %(new)d %(len)d" % case)
    lens, news = [], []
    for b in range(case["batch"]):
        new, length = case["new"], case["len"]
        if case["ragged"] and b:
            if new > 16:
                new = rng.randint(1, new)
            length = _log(rng, new, length)
        lens.append(length)
        news.append(new)
    return lens, news


# ---------------------------------------------------------------------------
# The 4-bit format: value = (code - 8) * scale, codes 1 .. 15, two to a byte (the even
# value in the low bits), a scale for each 32 values of a token's head.
# ---------------------------------------------------------------------------

def _scale(amax):
    """The smallest e5m2 number s >= 2^-14 with amax <= 7.5 s, as fp32."""
    m, e = torch.frexp(amax.double() / 7.5)
    s = torch.ceil(m * 8.0) * torch.exp2(e.double() - 3.0)
    return s.clamp(SCALE_MIN, SCALE_MAX).float()


def _coded(x):
    """x [..., dim] fp32 -> (codes [..., dim / 2] uint8, scales [..., dim / 32] e5m2)."""
    g = x.unflatten(-1, (-1, GROUP))
    s = _scale(torch.where(g.isfinite(), g.abs(), 0.0).amax(-1))
    q = torch.round(g / s[..., None]).clamp(-7, 7)
    c = (torch.where(q.isnan(), 0.0, q) + 8.0).to(torch.uint8).flatten(-2)
    s = torch.where(g.isnan().any(-1), math.nan, s)
    return c[..., 0::2] | c[..., 1::2] << 4, s.to(torch.float8_e5m2)


def _valued(codes, scales):
    """The fp32 values that codes and scales stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    return (c.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the limits (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875)
    return torch.where(amax > 0, e, EXP_MIN).clamp(EXP_MIN, EXP_MAX)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _pages_of(lens, page, width, gen):
    """Pages in scattered order, as a cache that has served for a while holds them; -1 past a sequence's end."""
    counts = [-(-n // page) for n in lens]
    total = sum(counts)
    ids = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    held = torch.arange(width, device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[held] = ids
    return table, total


def _image_positions(lens, news, axes):
    """Positions [tokens, axes]: of each sequence's new tokens a quarter text, then an image's patches in rows,
    then text that goes on behind the image's longer side."""
    parts = []
    for length, new in zip(lens, news):
        i, text = torch.arange(new), new // 4
        patches = new // 2
        wide = max(1, math.isqrt(max(patches - 1, 0)) + 1)
        at, begin = i - text, length - new
        inside, behind = (at >= 0) & (at < patches), at >= patches
        past = begin + text + wide + at - patches
        rows = torch.where(inside, begin + text + at // wide, torch.where(behind, past, begin + i))
        columns = torch.where(inside, begin + text + at % wide, torch.where(behind, past, begin + i))
        still = torch.where(inside, begin + text, torch.where(behind, past, begin + i))
        parts.append(torch.stack((still, rows, columns)[3 - axes:], 1))
    return torch.cat(parts).to(torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 6007 + 29)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    lens, news = _lengths(case)
    Hq, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    width = -(-max(lens) // P)
    table, total = _pages_of(lens, P, width, gen)
    T = sum(news)
    st = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_q=None, max_q=max(news))
    if min(news) != max(news):
        st["cu_q"] = torch.tensor([0] + news, device="cuda").cumsum(0).to(torch.int32)

    loud = torch.exp(normal(2, Hk, 1, D) * 0.7)                   # channels differ in size, keys' above all
    for i, name in enumerate(("k", "v")):
        x = normal(total, Hk, P, D) * (loud[i] if name == "k" else loud[i].sqrt())
        if case["op"] == "attention" or case["bits"] == 4:
            st[name + "_cache"], st[name + "_exp"] = _coded(x)
        else:
            e = _exponent(x.abs().amax((2, 3)))
            st[name + "_cache"] = (x * torch.exp2(-e.float())[..., None, None]).to(torch.float8_e4m3fn)
            st[name + "_exp"] = e.to(torch.int8)
    if case["op"] == "attention":
        sharp = torch.exp(normal(Hq, 1) * 0.5)                    # some heads look at few tokens, some at many
        st["q"] = (normal(T, Hq, D) * sharp).to(torch.bfloat16)
        return st
    qkv = normal(T, Hq + 2 * Hk, D)                               # the projection's output, q, k and v side by side
    qkv[:, Hq:Hq + Hk] *= loud[0, :, 0]
    qkv = qkv.to(torch.bfloat16)
    st["q"], st["k"], st["v"] = qkv.split([Hq, Hk, Hk], 1)
    half = case["rotary"] // 2
    # A rotation's frequency in turns per position, as a fraction of 2^64.
    st["turns"] = torch.tensor([int(500000.0 ** (-i / half) / (2 * math.pi) * 2.0 ** 64) for i in range(half)],
                               dtype=torch.int64, device="cuda")
    st["q_norm"] = st["k_norm"] = st["positions"] = st["axes"] = None
    if case["norm"]:
        st["q_norm"], st["k_norm"] = ((1.0 + 0.3 * normal(D)).to(torch.bfloat16) for _ in range(2))
    if case["axes"]:
        st["positions"] = _image_positions(lens, news, case["axes"])
        j = torch.arange(half, device="cuda")                     # pairs by turns, or in runs
        st["axes"] = (j % case["axes"] if case["interleaved"] else j * case["axes"] // half).to(torch.uint8)
    return st


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return {"attention": _own_attention, "kv_append": _own_append}[st["case"]["op"]](st)
    return {"attention": _plain_attention, "kv_append": _plain_append}[st["case"]["op"]](st)


def _own_attention(st):
    import bit_groupwise_weight_gb300 as lb
    q = st["q"]
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    out = lb.attention(q, st["k_cache"], st["v_cache"], st["k_exp"], st["v_exp"], st["table"], st["lens"],
                       cu_q=st["cu_q"], max_q=st["max_q"], window=st["case"]["window"], lse=lse)
    return {"out": out, "lse": lse}


def _own_append(st):
    import bit_groupwise_weight_gb300 as lb
    cache = st["k_cache"], st["v_cache"], st["k_exp"], st["v_exp"]
    q = lb.kv_append(st["q"], st["k"], st["v"], *cache, st["table"], st["lens"], cu_q=st["cu_q"], max_q=st["max_q"],
                     turns=st["turns"], interleaved=st["case"]["interleaved"], q_norm=st["q_norm"], k_norm=st["k_norm"],
                     eps=1e-6, positions=st["positions"], axes=st["axes"])
    if st["case"]["bits"] == 8:
        return {"q": q, "k_cache": cache[0], "v_cache": cache[1], "k_exp": cache[2], "v_exp": cache[3]}
    k, v = lb.cache_values(*cache)
    return {"q": q, "k": k, "v": v}


def _rows(st):
    """(sequence, position, place among the sequence's new tokens) of each new token."""
    T, lens = st["q"].shape[0], st["lens"].long()
    at, B = torch.arange(T, device=lens.device), lens.shape[0]
    if st["cu_q"] is None:
        n = T // B
        return at // n, lens[at // n] - n + at % n, at % n
    cu = st["cu_q"].long()
    seq = torch.searchsorted(cu[1:], at, right=True)
    return seq, lens[seq] - cu[seq + 1] + at, at - cu[seq]


def _plain_attention(st):
    c, table, lens, q = st["case"], st["table"].long().clamp(min=0), st["lens"].long(), st["q"]
    (B, W), (T, Hq, D) = table.shape, q.shape
    Hk, P, n = c["kv_heads"], c["page"], st["max_q"]
    G, L = Hq // Hk, W * P
    seq, pos, place = _rows(st)
    key = torch.arange(L, device=q.device)
    held = key[None] < lens[:, None]                                               # [B, L]

    def whole(name):                                                               # [B, Hk, L, D], zero past the end
        x = _valued(st[name + "_cache"][table], st[name + "_exp"].view(torch.uint8)[table].view(torch.float8_e5m2))
        x = x.transpose(1, 2).reshape(B, Hk, L, D)
        return torch.where(held[:, None, :, None], x, 0.0)

    qs = torch.zeros(B, n, Hq, D, device=q.device)
    qs[seq, place] = q.float()
    where = torch.full((B, n), -1, dtype=torch.int64, device=q.device)
    where[seq, place] = pos
    seen = held[:, None] & (key <= where[..., None])                               # [B, n, L]
    if c["window"]:
        seen = seen & (key > where[..., None] - c["window"])
    seen = seen[:, None, :, None].expand(B, Hk, n, G, L).reshape(B, Hk, n * G, L)
    qs = qs.reshape(B, n, Hk, G, D).transpose(1, 2).reshape(B, Hk, n * G, D)
    s = (qs @ whole("k").transpose(2, 3)) * (1.0 / math.sqrt(D))
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = torch.where(z > 0, (p @ whole("v")) / z, 0.0)
    lse = torch.log(z) + m
    o = o.reshape(B, Hk, n, G, D).transpose(1, 2).reshape(B, n, Hq, D)
    lse = lse.reshape(B, Hk, n, G).transpose(1, 2).reshape(B, n, Hq)
    return {"out": o[seq, place].to(torch.bfloat16), "lse": lse[seq, place]}


def _normed(x, weight):
    """x [T, heads, dim] fp32 over its root mean square, times weight.  The squares are added in pairs (neighbours,
    then neighbouring sums): codes next to a border need the same sum whoever adds it."""
    if weight is None:
        return x
    s = x * x
    while s.shape[-1] > 1:
        s = s[..., 0::2] + s[..., 1::2]
    return x * (1.0 / torch.sqrt(s * (1.0 / x.shape[-1]) + 1e-6)) * weight.float()


def _rotated(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, x[..., R:]), -1)


def _plain_append(st):
    c, table = st["case"], st["table"].long()
    P = c["page"]
    seq, pos, place = _rows(st)
    turned = pos[:, None] if st["positions"] is None else st["positions"].long()[:, st["axes"].long()]
    phase = turned * st["turns"]                                                   # whole turns wrap around
    angle = (phase >> 32).float() * (2 * math.pi * 2.0 ** -32)
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    page, slot = table[seq, pos // P], pos % P
    q = _rotated(_normed(st["q"].float(), st["q_norm"]), cos, sin, c["interleaved"]).to(torch.bfloat16)
    k, v = _rotated(_normed(st["k"].float(), st["k_norm"]), cos, sin, c["interleaved"]), st["v"].float()
    if c["bits"] == 4:
        out = {"q": q}
        for name, x in (("k", k), ("v", v)):
            codes, scales = st[name + "_cache"], st[name + "_exp"]
            new, s = _coded(x)
            codes[page, :, slot] = new
            scales.view(torch.uint8)[page, :, slot] = s.view(torch.uint8)
            out[name] = _valued(codes, scales).to(torch.bfloat16)
        return out
    pages = st["k_cache"].shape[0]
    # The page in which each sequence's new tokens begin, where older tokens are in it too.
    first = place == 0
    older = torch.where(first, slot, 0)
    for name, x in (("k", k), ("v", v)):
        codes, exps = st[name + "_cache"].view(torch.uint8), st[name + "_exp"]
        size = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)                    # [T, Hk]
        amax = torch.zeros(pages, size.shape[1], device=x.device)
        amax.scatter_reduce_(0, page[:, None].expand_as(size), size, "amax")
        old = exps[page].int()
        need = _exponent(amax)[page]
        shared = torch.zeros(pages, dtype=torch.bool, device=x.device)
        shared[page[older > 0]] = True
        e = torch.where(shared[page][:, None], torch.maximum(need, old), need)
        # Older tokens of a page whose scale has grown are rounded to it.
        was = codes[page[first]].view(torch.float8_e4m3fn).float()
        scaled = (was * torch.exp2((old - e)[first].float())[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        keep = torch.arange(P, device=x.device) < older[first][:, None]
        codes[page[first]] = torch.where(keep[:, None, :, None], scaled, codes[page[first]])
        exps[page] = e.to(torch.int8)
        x = (x * torch.exp2(-e.float())[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
        codes[page, :, slot] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"], "k_exp": st["k_exp"], "v_exp": st["v_exp"]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    lens, news = _lengths(case)
    Hq, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    T = sum(news)
    coded = D // 2 + D // GROUP                                                    # bytes of a token's head in 4 bits
    if case["op"] == "kv_append":
        rows = T * (Hq + Hk) * D
        moved = T * D * (4 * Hq + 4 * Hk) + 4 * T * case["axes"] + 8 * len(lens)   # q, k, v read, q written
        if case["bits"] == 4:                                                      # the codes written, the cache read as values
            moved += 2 * Hk * (T * coded + sum(-(-n // P) for n in lens) * P * (coded + 2 * D))
        else:
            moved += 2 * Hk * (T * D + sum((n - 1) // P - (n - m) // P + 1 for n, m in zip(lens, news)))
        return {"bytes": moved, "flops": T * (Hq + Hk) * case["rotary"] * 3 + (4 * rows if case["norm"] else 0) + 4 * T * Hk * D}
    w = case["window"] or 1 << 40
    keys = sum(min(n, w + m - 1) for n, m in zip(lens, news))
    pairs = sum(min(p + 1, w) for n, m in zip(lens, news) for p in range(n - m, n))
    return {"bytes": 4 * T * Hq * D + 4 * T * Hq + 2 * keys * Hk * coded + 4 * (keys // P), "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"attention": _exact_attention, "kv_append": _exact_append}[case["op"]](st)


def _each(st):
    """For each sequence: its pages, its length, and which rows of q are its."""
    end = 0
    for b, (length, new) in enumerate(zip(*_lengths(st["case"]))):
        start, end = end, end + new
        pages = st["table"][b, :-(-length // st["case"]["page"])].long()
        yield pages, length, new, slice(start, end)


def _exact_values(codes, scales):
    """fp64 values of 4-bit codes: the even value of a byte is its low half."""
    x = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = codes.bitwise_and(15).double() - 8, codes.bitwise_right_shift(4).double() - 8
    return x * scales.to(torch.float32).double().repeat_interleave(GROUP, -1)


def _exact_attention(st):
    c, q = st["case"], st["q"].double()
    G = c["heads"] // c["kv_heads"]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    for pages, length, new, rows in _each(st):
        pos = torch.arange(length - new, length, device=q.device)[:, None]
        key = torch.arange(length, device=q.device)[None]
        hidden = key > pos
        if c["window"]:
            hidden = hidden | (key <= pos - c["window"])
        for h in range(c["kv_heads"]):
            k, v = (_exact_values(st[x + "_cache"][pages, h], st[x + "_exp"].view(torch.uint8)[pages, h].view(torch.float8_e5m2))
                    .reshape(-1, c["dim"])[:length] for x in "kv")
            for g in range(h * G, h * G + G):
                s = (q[rows, g] @ k.T / math.sqrt(c["dim"])).masked_fill(hidden, -math.inf)
                out[rows, g] = torch.softmax(s, -1) @ v
                lse[rows, g] = torch.logsumexp(s, -1)
    return {"out": out, "lse": lse}


def _exact_rows(st, name, rows, pos):
    """A sequence's rows of q, k or v in 64 bits, normed and turned."""
    x = st[name][rows].double()
    if name == "v":
        return x
    if st[name + "_norm"] is not None:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * st[name + "_norm"].double()
    half = st["turns"].shape[0]
    p = pos[:, None] if st["positions"] is None else st["positions"][rows].long().gather(1, st["axes"].long().expand(len(pos), half))
    angle = (p * st["turns"]).double()[:, None] * (2 * math.pi / 2.0 ** 64)
    i = torch.arange(half, device=x.device)
    i, j = (2 * i, 2 * i + 1) if st["case"]["interleaved"] else (i, i + half)
    y = x.clone()
    y[..., i], y[..., j] = x[..., i] * angle.cos() - x[..., j] * angle.sin(), x[..., j] * angle.cos() + x[..., i] * angle.sin()
    return y


def _exact_append(st):
    c = st["case"]
    P, names = c["page"], ("k", "v")
    q_out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    if c["bits"] == 4:
        held = {x: _exact_values(st[x + "_cache"], st[x + "_exp"]) for x in names}
    else:
        held = {x: st[x + "_cache"].to(torch.float32).double() for x in names}
    exps = {x: st[x + "_exp"].clone() for x in names}
    grid = torch.tensor([m * 2.0 ** e for e in range(-16, 14) for m in (4, 5, 6, 7)], dtype=torch.float64, device="cuda")
    for pages, length, new, rows in _each(st):
        pos = torch.arange(length - new, length, device="cuda")
        q_out[rows] = _exact_rows(st, "q", rows, pos)
        for x in names:
            fresh = _exact_rows(st, x, rows, pos)
            if c["bits"] == 4:
                g = fresh.reshape(new, c["kv_heads"], -1, GROUP)
                s = grid[torch.searchsorted(grid, g.abs().amax(-1) / 7.5).clamp(max=len(grid) - 1)][..., None]
                held[x][pages[pos // P], :, pos % P] = (torch.round(g / s).clamp(-7, 7) * s).flatten(-2)
                continue
            for at in range((length - new) // P, -(-length // P)):
                lo, hi = max(at * P, length - new), min(at * P + P, length)
                part, page = fresh[lo - length + new:hi - length + new].transpose(0, 1), pages[at]    # [Hk, tokens, D]
                amax = part.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(EXP_MIN, EXP_MAX)
                e = (e - (amax <= E4M3_MAX * 2.0 ** (e - 1)).double()).clamp(EXP_MIN)      # where log2 came out too large
                if lo > at * P:
                    was = exps[x][page].double()
                    e = torch.maximum(e, was)
                    kept = held[x][page, :, :lo - at * P] * 2.0 ** (was - e)[:, None, None]
                    held[x][page, :, :lo - at * P] = kept.float().to(torch.float8_e4m3fn).to(torch.float32).double()
                exps[x][page] = e.to(torch.int8)
                part = part * 2.0 ** -e[:, None, None]
                held[x][page, :, lo - at * P:hi - at * P] = part.float().to(torch.float8_e4m3fn).to(torch.float32).double()
    if c["bits"] == 4:
        return {"q": q_out, "k": held["k"], "v": held["v"]}
    return {"q": q_out, "k_cache": held["k"], "v_cache": held["v"], "k_exp": exps["k"], "v_exp": exps["v"]}
