"""Plain 64-bit definitions of the decoder operators (cache append, attention over the
8-bit cache, sampling) for the tests, on the CPU in numpy, and seeded inputs.

Nothing here uses the library: e4m3 values come from their definition, rotations from
Python's integers and fp64, attention from explicit masks, sampling from a sort."""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

E4M3 = np.array([(m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)) if (e, m) != (15, 7) else np.nan
                 for e in range(16) for m in range(8)])
E4M3 = np.concatenate([E4M3, -E4M3])                      # value of every code
GRID = E4M3[:127]                                         # 0 .. 448
EXP_MIN, EXP_MAX = -64, 64


def e4m3_round(x):
    """Codes of the nearest e4m3 values (ties to the even code), past 448 clamped; x fp64."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(GRID, a), 1, 126)
    lo = hi - 1
    up = (a - GRID[lo] > GRID[hi] - a) | ((a - GRID[lo] == GRID[hi] - a) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | (np.signbit(x) & ~np.isnan(x)).astype(np.uint8) << 7).astype(np.uint8)


def page_exponent(amax: float) -> int:
    e = EXP_MIN
    while e < EXP_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


@dataclasses.dataclass
class Batch:
    """Sequences over a cache, on the CPU: codes [pages, heads, page, dim] uint8."""
    lens: list
    news: list
    table: np.ndarray
    k: np.ndarray
    v: np.ndarray
    k_exp: np.ndarray
    v_exp: np.ndarray

    @property
    def page(self):
        return self.k.shape[2]

    @property
    def starts(self):
        return np.concatenate([[0], np.cumsum(self.news)])

    def device(self, uniform: bool | None = None):
        """(cache tensors, page_table, lens, cu_q or None) on the GPU."""
        cache = tuple(torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in (self.k, self.v)) + tuple(
            torch.from_numpy(e).cuda() for e in (self.k_exp, self.v_exp))
        table = torch.from_numpy(self.table).cuda()
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        same = len(set(self.news)) <= 1 if uniform is None else uniform
        cu = None if same else torch.from_numpy(self.starts.astype(np.int32)).cuda()
        return cache, table, lens, cu


def make_batch(seed, lens, news, heads, dim, page, *, garbage=True, spare=2, exps=(-4, 3)) -> Batch:
    """A cache whose pages are scattered; unused slots and spare pages hold NaN codes."""
    rng = np.random.default_rng([seed, heads, dim, page, len(lens)])
    counts = [-(-n // page) for n in lens]
    pages, width = sum(counts) + spare, max(max(counts), 1)
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    codes = []
    for _ in range(2):
        c = e4m3_round(np.clip(rng.standard_normal((pages, heads, page, dim)) * 60, -448, 448))
        if garbage:
            used = np.zeros((pages, page), bool)
            for b, n in enumerate(lens):
                for i in range(n):
                    used[table[b, i // page], i % page] = True
            c = np.where(used[:, None, :, None], c, np.uint8(0xFF)).astype(np.uint8)
        codes.append(c)
    e = [rng.integers(exps[0] - 6, exps[1] - 6, (pages, heads)).astype(np.int8) for _ in range(2)]
    return Batch(list(lens), list(news), table, codes[0], codes[1], e[0], e[1])


def cached(b: Batch, seq: int, head: int, which: str):
    """fp64 [len, dim] of a sequence's keys or values of one head."""
    codes, exps = (b.k, b.k_exp) if which == "k" else (b.v, b.v_exp)
    n = b.lens[seq]
    ids = b.table[seq, :-(-n // b.page)].astype(np.int64) if n else np.zeros(0, np.int64)
    inside = (ids >= 0) & (ids < codes.shape[0])
    safe = np.where(inside, ids, 0)
    x = E4M3[codes[safe, head]] * (2.0 ** exps[safe, head].astype(np.float64))[:, None, None]
    x = np.where(inside[:, None, None], x, 0.0)
    return x.reshape(-1, codes.shape[3])[:n]


def attention(q: np.ndarray, b: Batch, scale: float, window: int = 0):
    """(out, lse, bound, lse_bound): q fp64 [T, heads, dim].

    The bounds on |kernel - out| follow from the kernel's arithmetic: scores summed in
    fp32 (a few units of the magnitude sum, 2^-20 of it), 2^x to 2^-22, weights held
    as fp16 (2^-11 of themselves, or 2^-24 of the largest weight times page scale),
    and one rounding to bf16 (2^-8 of the value covers it with its half unit)."""
    T, heads, dim = q.shape
    group = heads // b.k.shape[1]
    out, bound = np.zeros_like(q), np.zeros_like(q)
    lse, lse_bound = np.full((T, heads), -np.inf), np.zeros((T, heads))
    for s, n in enumerate(b.news):
        rows = slice(b.starts[s], b.starts[s] + n)
        pos = b.lens[s] - n + np.arange(n)[:, None]
        t = np.arange(b.lens[s])[None]
        seen = t <= pos
        if window:
            seen &= t > pos - window
        ids = np.clip(b.table[s], 0, b.k.shape[0] - 1)
        for h in range(heads):
            k, v = cached(b, s, h // group, "k"), cached(b, s, h // group, "v")
            x = np.where(seen, q[rows, h] @ np.nan_to_num(k).T * scale, -np.inf)
            with np.errstate(invalid="ignore"):
                x = np.where(seen & np.isnan(k).any(1)[None], np.nan, x)
            m = np.where(seen.any(1, keepdims=True), np.max(np.where(seen, x, -np.inf), 1, keepdims=True, initial=-np.inf), 0.0)
            m = np.where(np.isinf(m), 0.0, m)
            w = np.where(seen, np.exp(x - m), 0.0)
            z = w.sum(1, keepdims=True)
            p = np.divide(w, z, out=np.zeros_like(w), where=z != 0)
            o = p @ np.nan_to_num(v)
            o = np.where((seen.astype(float) @ np.isnan(v).astype(float)) > 0, np.nan, o)
            out[rows, h] = np.where(np.isnan(z), np.nan, o)
            with np.errstate(divide="ignore"):
                lse[rows, h] = (np.log(z) + m)[:, 0]
            scales = np.repeat(b.v_exp[ids, h // group].astype(np.float64), b.page)[:b.lens[s]]
            av = np.abs(np.nan_to_num(v))
            mag = np.abs(q[rows, h]) @ np.abs(np.nan_to_num(k)).T * scale                 # of the score sums
            d = np.where(seen, mag * 2.0 ** -20 + np.abs(np.nan_to_num(x, neginf=0.0)) * 2.0 ** -20 + 2.0 ** -20, 0.0)
            top = np.max(p * 2.0 ** scales[None, :], 1, keepdims=True, initial=0.0)
            codes = av * 2.0 ** -scales[:, None]
            rel = d + np.max(d, 1, keepdims=True, initial=0.0) + 2.0 ** -11
            bound[rows, h] = 2.0 ** -8 * np.abs(np.nan_to_num(o)) + (p * rel) @ av + 2.0 ** -24 * top * (seen.astype(float) @ codes) + 1e-30
            lse_bound[rows, h] = 2.0 * np.max(d, 1, initial=0.0) + 2.0 ** -21 * np.abs(np.nan_to_num(lse[rows, h], neginf=0.0)) + 2.0 ** -18
    return out, lse, bound, lse_bound


def angles(positions, turns):
    """fp64 [tokens, pairs], from the wrapped 64-bit phase."""
    ph = [[((int(p) * int(t) + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64 for t in turns] for p in positions]
    return 2 * math.pi * np.array(ph).reshape(len(positions), len(turns))


def rotate(x, positions, turns, interleaved, factor):
    """fp64 [tokens, heads, dim] rotated, and the magnitude |a| + |b| behind each value."""
    R = 2 * len(turns)
    out, mag = x.copy(), np.abs(x)
    if R:
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
        th = angles(positions, turns)[:, None]
        c, s = np.cos(th) * factor, np.sin(th) * factor
        y, z, g = a * c - b * s, a * s + b * c, (np.abs(a) + np.abs(b)) * factor
        if interleaved:
            out[..., 0:R:2], out[..., 1:R:2] = y, z
            mag[..., 0:R:2] = mag[..., 1:R:2] = g
        else:
            out[..., :R // 2], out[..., R // 2:R] = y, z
            mag[..., :R // 2] = mag[..., R // 2:R] = g
    return out, mag


def weights(row: np.ndarray, temperature: float):
    """(s, W as floats of whole numbers, bound on each W's error): row fp64."""
    m = row.max()
    with np.errstate(invalid="ignore"):
        s = np.where(row == m, 0.0, (row - m) / np.float64(temperature))
    w = np.exp(s)
    # s is off by 2^-23 of itself (a difference and a product in fp32, 1/T rounded), expf by 2 units.
    with np.errstate(invalid="ignore"):
        err = np.nan_to_num(w * (np.abs(s) * 2.0 ** -22 + 2.0 ** -22)) * 2.0 ** 30 + (w > 0) * 0.5
    return s, np.rint(w * 2.0 ** 30), err


def check_sample(row, u, temperature, top_k, top_p, min_p, token, logprob):
    """Asserts that `token` is a draw of the definition, allowing each weight its error."""
    row = np.where(np.isnan(row), -np.inf, row)
    if not (row > -np.inf).any():
        assert token == -1 and logprob == -np.inf
        return
    if not temperature > 0:
        assert token == int(np.argmax(row)) and logprob == 0.0
        return
    s, W, err = weights(row, temperature)
    order = np.argsort(-row, kind="stable")
    kept = order if top_k <= 0 else order[:top_k]
    w = np.exp(s)
    sure = kept[w[kept] >= min(min_p, 1.0) + 2.0 ** -20] if min_p > 0 else kept
    kept = kept[w[kept] >= min(min_p, 1.0) - 2.0 ** -20] if min_p > 0 else kept
    before = np.cumsum(W[kept]) - W[kept]
    slack = err[kept].sum() + W[kept].sum() - W[sure].sum()
    limit = max(1.0, math.ceil(top_p * W[kept].sum())) if top_p < 1 else np.inf
    loose, tight = kept[before < limit + slack], kept[before < max(limit - slack, 1.0)]
    assert token in loose, f"token {token} is not among the kept"
    lo_total, hi_total = W[tight].sum() - slack, W[loose].sum() + slack
    asc_l, asc_t = np.sort(loose), np.sort(tight)
    upto = W[asc_l[asc_l <= token]].sum() + slack                     # most that can come up to the token
    ahead = W[asc_t[asc_t < token]].sum() - slack                     # least that must come before it
    assert upto > math.floor(u * lo_total) - 1 and ahead <= u * hi_total, f"token {token} is not the draw"
    assert abs(logprob - (s[token] - math.log(W[tight].sum() / 2.0 ** 30))) <= (
        abs(s[token]) * 2.0 ** -21 + 2.0 ** -20 + (hi_total - lo_total) / W[tight].sum())
