"""Cases of the operators between the low-bit linear layers of a decoder: what a decode
step does from the qkv projection's output to the output projection's input, and from
the last logits to the next token.

kv_append   rotary positions on q and k, and the new keys and values written into a
            paged cache of 8-bit floats (e4m3) with one power-of-two scale for each
            page of tokens and head.
attention   softmax attention of the new tokens' queries over that cache.
sample      a token for each row of logits: temperature, top-k, min-p, top-p, from
            given random numbers.

`run` computes them with elementary torch operations, or, where `own` is true, calls
the library's operators.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -64, 64            # limits of a page's scale exponent
UNIT = 2.0 ** 30                      # a sampling weight of 1, in fixed point


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One user, short prompt: latency is all there is (heads of an 8B decoder).
        dict(name="attn-decode-1", op="attention", batch=1, new=1, len=257, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # One user at the end of a long document: the cache is read once, 8 key-value heads.
        dict(name="attn-decode-long", op="attention", batch=1, new=1, len=131001, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # A serving batch whose sequences have very different lengths.
        dict(name="attn-decode-batch", op="attention", batch=48, new=1, len=8192, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # Heads of a 1B decoder, small pages, a sliding window that cuts most pages off.
        dict(name="attn-decode-window", op="attention", batch=96, new=1, len=3001, ragged=True,
             heads=32, kv_heads=8, dim=64, page=16, window=1000),
        # Checking five guessed tokens a sequence at once (heads of a 3B decoder, 3 per kv head).
        dict(name="attn-verify", op="attention", batch=8, new=5, len=6001, ragged=True,
             heads=24, kv_heads=8, dim=128, page=64, window=0),
        # A whole prompt.
        dict(name="attn-prefill", op="attention", batch=1, new=4096, len=4096, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # Chunks of several prompts behind what is cached of them already.
        dict(name="attn-chunk", op="attention", batch=4, new=701, len=9001, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, window=0),
        # A decode step of one user: one token's rotation and cache write.
        dict(name="append-decode-1", op="kv_append", batch=1, new=1, len=1000, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, rotary=128, interleaved=False),
        # A whole prompt's keys and values, half of each head rotated, pairs interleaved.
        dict(name="append-prefill", op="kv_append", batch=2, new=8001, len=8001, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, rotary=64, interleaved=True),
        # One user's next token, bf16 logits as the output layer leaves them.
        dict(name="sample-1", op="sample", batch=1, vocab=128256, dtype="bfloat16", filters="mixed"),
        # A serving batch, nucleus sampling.
        dict(name="sample-64", op="sample", batch=64, vocab=128256, dtype="bfloat16", filters="nucleus"),
        # A large batch where every row has settings of its own, 32-bit logits.
        dict(name="sample-256", op="sample", batch=256, vocab=128256, dtype="float32", filters="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "kv_append", "sample"])
    if op == "sample":
        batch = _log(rng, 1, 256)
        vocab = _log(rng, 1000, min(200000, 256 * 128256 // batch))
        return dict(op=op, batch=batch, vocab=vocab, dtype=rng.choice(["bfloat16", "float32", "float16"]),
                    filters=rng.choice(["plain", "nucleus", "mixed"]))
    heads, kv_heads = rng.choice([(32, 8), (24, 8), (32, 8), (16, 16), (40, 8), (16, 2), (16, 1)])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    if op == "kv_append":
        batch = _log(rng, 1, 64)
        new = rng.choice([1, _log(rng, 1, 16002 // batch)])
        return dict(op=op, batch=batch, new=new, len=new + _log(rng, 1, 4000) - 1, ragged=rng.random() < 0.5,
                    heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    rotary=rng.choice([dim, dim // 2, dim // 4 * 3, 10]), interleaved=rng.random() < 0.5)
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
# Inputs
# ---------------------------------------------------------------------------

def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the limits (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875)
    return torch.where(amax > 0, e, EXP_MIN).clamp(EXP_MIN, EXP_MAX)


def _pages_of(lens, page, width, gen):
    """Pages in scattered order, as a cache that has served for a while holds them; -1 past a sequence's end."""
    counts = [-(-n // page) for n in lens]
    total = sum(counts)
    ids = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    held = torch.arange(width, device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[held] = ids
    return table, total


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 11)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "sample":
        B, V = case["batch"], case["vocab"]
        logits = normal(B, V) * 2.2
        peaks = torch.randint(0, V, (B, 12), generator=gen, device="cuda")
        logits.scatter_add_(1, peaks, 6 + 3 * normal(B, 12))       # a few likely tokens over a broad tail

        def pick(values):
            at = torch.randint(0, len(values), (B,), generator=gen, device="cuda")
            return torch.tensor(values, device="cuda")[at]
        st = dict(case=case, logits=logits.to(getattr(torch, case["dtype"])),
                  u=torch.rand(B, generator=gen, device="cuda"),
                  temperature=pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.3]),
                  top_k=torch.zeros(B, dtype=torch.int32, device="cuda"),
                  top_p=torch.ones(B, device="cuda"), min_p=torch.zeros(B, device="cuda"))
        if case["filters"] == "nucleus":
            st["temperature"] = pick([0.6, 0.8, 1.0])
            st["top_p"] = pick([0.8, 0.9, 0.95])
        elif case["filters"] == "mixed":
            st["top_k"] = pick([0, 0, 1, 20, 50, 400]).to(torch.int32)
            st["top_p"] = pick([1.0, 0.7, 0.9, 0.95, 0.99])
            st["min_p"] = pick([0.0, 0.0, 0.02, 0.1])
        return st

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
        e = _exponent(x.abs().amax((2, 3)))
        st[name + "_cache"] = (x * torch.exp2(-e.float())[..., None, None]).to(torch.float8_e4m3fn)
        st[name + "_exp"] = e.to(torch.int8)
    if case["op"] == "attention":
        sharp = torch.exp(normal(Hq, 1) * 0.5)                    # some heads look at few tokens, some at many
        st["q"] = (normal(T, Hq, D) * sharp).to(torch.bfloat16)
    else:
        qkv = normal(T, Hq + 2 * Hk, D)                           # the projection's output, q, k and v side by side
        qkv[:, Hq:Hq + Hk] *= loud[0, :, 0]
        qkv = qkv.to(torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv.split([Hq, Hk, Hk], 1)
        R = case["rotary"]
        # A rotation's frequency in turns per position, as a fraction of 2^64.
        st["turns"] = torch.tensor([int(500000.0 ** (-2.0 * i / R) / (2 * math.pi) * 2.0 ** 64) for i in range(R // 2)],
                                   dtype=torch.int64, device="cuda")
        st["factor"] = 1.0
    return st


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"attention": _own_attention, "kv_append": _own_append, "sample": _own_sample}[op](st)
    return {"attention": _plain_attention, "kv_append": _plain_append, "sample": _plain_sample}[op](st)


def _own_attention(st):
    import bit_groupwise_weight_gb300 as lb
    q = st["q"]
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    out = lb.attention(q, st["k_cache"], st["v_cache"], st["k_exp"], st["v_exp"], st["table"], st["lens"],
                       cu_q=st["cu_q"], max_q=st["max_q"], window=st["case"]["window"], lse=lse)
    return {"out": out, "lse": lse}


def _own_append(st):
    import bit_groupwise_weight_gb300 as lb
    q = lb.kv_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["k_exp"], st["v_exp"], st["table"],
                     st["lens"], cu_q=st["cu_q"], max_q=st["max_q"], turns=st["turns"],
                     interleaved=st["case"]["interleaved"], factor=st["factor"])
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"], "k_exp": st["k_exp"], "v_exp": st["v_exp"]}


def _own_sample(st):
    import bit_groupwise_weight_gb300 as lb
    logprob = torch.empty(st["u"].shape, dtype=torch.float32, device=st["u"].device)
    token = lb.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                      min_p=st["min_p"], logprob=logprob)
    return {"token": token, "logprob": logprob}


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
        x = st[name + "_cache"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(st[name + "_exp"][table].float())[..., None, None]
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


def _rotated(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    x = x.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, x[..., R:]), -1)


def _plain_append(st):
    c, table, lens = st["case"], st["table"].long(), st["lens"].long()
    P, pages = c["page"], st["k_cache"].shape[0]
    seq, pos, place = _rows(st)
    phase = pos[:, None] * st["turns"]                                             # whole turns wrap around
    angle = (phase >> 32).float() * (2 * math.pi * 2.0 ** -32)
    cos, sin = (torch.cos(angle) * st["factor"])[:, None], (torch.sin(angle) * st["factor"])[:, None]
    page = table[seq, pos // P]
    # The page in which each sequence's new tokens begin, where older tokens are in it too.
    first = place == 0
    older = torch.where(first, pos % P, 0)
    for name, x in (("k", _rotated(st["k"], cos, sin, c["interleaved"])), ("v", st["v"].float())):
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
        codes[page, :, pos % P] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    q = _rotated(st["q"], cos, sin, c["interleaved"]).to(torch.bfloat16)
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"], "k_exp": st["k_exp"], "v_exp": st["v_exp"]}


def _plain_sample(st):
    x = st["logits"].float()
    B, V = x.shape
    x = torch.where(x.isnan(), -math.inf, x)
    top, best = x.max(-1, keepdim=True)
    t = st["temperature"][:, None]
    s = (x - top) * torch.where(t > 0, 1.0 / t, 1.0)
    w = torch.exp(s)
    units = torch.round(w * UNIT).long()                                           # weights in fixed point: sums are exact
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices            # ties: lowest index first
    rank = torch.arange(V, device=x.device)
    k = st["top_k"].long()[:, None]
    kept = ((k <= 0) | (rank < k)) & (w >= st["min_p"][:, None]).gather(1, order)
    mass = torch.where(kept, units.gather(1, order), 0)
    limit = torch.ceil(st["top_p"].double()[:, None] * mass.sum(-1, keepdim=True)).long().clamp(min=1)
    mass = torch.where(mass.cumsum(-1) - mass < limit, mass, 0)
    mass = torch.zeros_like(mass).scatter_(1, order, mass)                         # back to the tokens' own order
    total = mass.sum(-1, keepdim=True)
    target = torch.floor(st["u"].double()[:, None] * total).long()
    token = (mass.cumsum(-1) > target).to(torch.uint8).argmax(-1, keepdim=True)
    logprob = s.gather(1, token) - torch.log(total.float() / UNIT)
    best = torch.eq(x, top).to(torch.uint8).argmax(-1, keepdim=True)
    token, logprob = torch.where(t > 0, token, best), torch.where(t > 0, logprob, 0.0)
    return {"token": token[:, 0], "logprob": logprob[:, 0]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "sample":
        n = case["batch"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "float32" else 2) + case["batch"] * 32, "flops": 4 * n}
    lens, news = _lengths(case)
    Hq, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    T = sum(news)
    if case["op"] == "kv_append":
        pages = sum((n - 1) // P - (n - m) // P + 1 for n, m in zip(lens, news))
        return {"bytes": T * D * (4 * Hq + 6 * Hk) + 2 * Hk * pages + 8 * len(lens), "flops": T * (Hq + Hk) * case["rotary"] * 3 + 4 * T * Hk * D}
    w = case["window"] or 1 << 40
    keys = sum(min(n, w + m - 1) for n, m in zip(lens, news))
    pairs = sum(min(p + 1, w) for n, m in zip(lens, news) for p in range(n - m, n))
    return {"bytes": 4 * T * Hq * D + 4 * T * Hq + 2 * keys * Hk * D + 2 * Hk * (keys // P) + 4 * (keys // P),
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"attention": _exact_attention, "kv_append": _exact_append, "sample": _exact_sample}[case["op"]](st)


def _each(st):
    """For each sequence: its pages, its length, and which rows of q are its."""
    end = 0
    for b, (length, new) in enumerate(zip(*_lengths(st["case"]))):
        start, end = end, end + new
        pages = st["table"][b, :-(-length // st["case"]["page"])].long()
        yield pages, length, new, slice(start, end)


def _values(codes, exps):
    return codes.to(torch.float32).double() * 2.0 ** exps.double()[..., None, None]


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
            k, v = (_values(st[x + "_cache"].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn), st[x + "_exp"][pages, h])
                    .reshape(-1, c["dim"])[:length] for x in "kv")
            for g in range(h * G, h * G + G):
                s = (q[rows, g] @ k.T / math.sqrt(c["dim"])).masked_fill(hidden, -math.inf)
                out[rows, g] = torch.softmax(s, -1) @ v
                lse[rows, g] = torch.logsumexp(s, -1)
    return {"out": out, "lse": lse}


def _exact_append(st):
    c = st["case"]
    P, half = c["page"], c["rotary"] // 2
    names = ("k", "v")
    codes = {x: st[x + "_cache"].to(torch.float32).double() for x in names}
    exps = {x: st[x + "_exp"].clone() for x in names}
    q_out = st["q"].double().clone()

    def turned(x, cos, sin):
        x = x.double().clone()
        i = torch.arange(half, device=x.device)
        i, j = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        x[..., i], x[..., j] = x[..., i] * cos - x[..., j] * sin, x[..., j] * cos + x[..., i] * sin
        return x

    for pages, length, new, rows in _each(st):
        pos = torch.arange(length - new, length, device=q_out.device)
        angle = (pos[:, None] * st["turns"]).double() * (2 * math.pi / 2.0 ** 64)
        cos, sin = torch.cos(angle)[:, None] * st["factor"], torch.sin(angle)[:, None] * st["factor"]
        q_out[rows] = turned(st["q"][rows], cos, sin)
        fresh = {"k": turned(st["k"][rows], cos, sin), "v": st["v"][rows].double()}
        for x in names:
            for at in range((length - new) // P, -(-length // P)):
                lo, hi = max(at * P, length - new), min(at * P + P, length)
                part, page = fresh[x][lo - length + new:hi - length + new].transpose(0, 1), pages[at]    # [Hk, tokens, D]
                amax = part.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(EXP_MIN, EXP_MAX)
                e = (e - (amax <= E4M3_MAX * 2.0 ** (e - 1)).double()).clamp(EXP_MIN)      # where log2 came out too large
                if lo > at * P:
                    was = exps[x][page].double()
                    e = torch.maximum(e, was)
                    kept = codes[x][page, :, :lo - at * P] * 2.0 ** (was - e)[:, None, None]
                    codes[x][page, :, :lo - at * P] = kept.float().to(torch.float8_e4m3fn).to(torch.float32).double()
                exps[x][page] = e.to(torch.int8)
                part = part * 2.0 ** -e[:, None, None]
                codes[x][page, :, lo - at * P:hi - at * P] = part.float().to(torch.float8_e4m3fn).to(torch.float32).double()
    return {"q": q_out, "k_cache": codes["k"], "v_cache": codes["v"], "k_exp": exps["k"], "v_exp": exps["v"]}


def _exact_sample(st):
    x = st["logits"].double()
    token, logprob = [], []
    for b in range(x.shape[0]):
        t, k, p, low = (float(st[n][b]) for n in ("temperature", "top_k", "top_p", "min_p"))
        row = x[b]
        s = (row - row.max()) / (t if t > 0 else 1.0)
        w = torch.round(torch.exp(s) * UNIT)
        by = torch.argsort(row, descending=True, stable=True)
        if t <= 0:
            token.append(int(by[0]))
            logprob.append(0.0)
            continue
        by = by[:int(k)] if k > 0 else by
        by = by[torch.exp(s[by]) >= low]
        limit = max(1.0, math.ceil(p * float(w[by].sum())))
        before = torch.cumsum(w[by], 0) - w[by]
        by = torch.sort(by[before < limit]).values
        total = torch.cumsum(w[by], 0)
        at = by[torch.searchsorted(total, torch.floor(st["u"][b].double() * total[-1]), right=True)]
        token.append(int(at))
        logprob.append(float(s[at]) - math.log(float(total[-1]) / UNIT))
    return {"token": torch.tensor(token), "logprob": torch.tensor(logprob, dtype=torch.float64)}
