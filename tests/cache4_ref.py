"""Plain 64-bit definitions of the 4-bit cache (its format, the write into it with head norms
and positions of several axes, attention over it) for the tests, on the CPU in numpy, and
seeded inputs.  Nothing here uses the library."""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

import decoder_ref as ref

GROUP = 32
E5M2 = np.array([(m / 4.0 * 2.0 ** -14 if e == 0 else (1 + m / 4.0) * 2.0 ** (e - 15)) if e < 31 else (np.inf if m == 0 else np.nan)
                 for e in range(32) for m in range(4)])
E5M2 = np.concatenate([E5M2, -E5M2])                      # value of every byte
SCALES = E5M2[4:124]                                      # what is written: 2^-14 .. 57344


def scale_byte(amax):
    """Byte of the smallest scale s with amax <= 7.5 s, the largest where there is none."""
    return 4 + np.minimum(np.searchsorted(SCALES * 7.5, amax), len(SCALES) - 1)


def coded(x):
    """x fp64 [..., dim] -> (codes [..., dim] 0 .. 15, scale bytes [..., dim / 32])."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    byte = scale_byte(np.where(np.isfinite(g), np.abs(g), 0.0).max(-1))
    q = np.clip(np.rint(g / E5M2[byte][..., None]), -7, 7)
    byte = np.where(np.isnan(g).any(-1), 0x7F, byte)
    return (np.nan_to_num(q) + 8).astype(np.uint8).reshape(x.shape), byte.astype(np.uint8)


def values(codes, scales):
    """fp64 values of unpacked codes and scale bytes; NaN where a scale is infinite or none."""
    s = np.where(np.isfinite(E5M2[scales]), E5M2[scales], np.nan)
    return (codes.astype(np.float64) - 8) * np.repeat(s, GROUP, -1)


def packed(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def unpacked(bytes_):
    out = np.empty(bytes_.shape[:-1] + (2 * bytes_.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = bytes_ & 15, bytes_ >> 4
    return out


@dataclasses.dataclass
class Batch:
    """Sequences over a cache, on the CPU: codes [pages, heads, page, dim], one to a byte, scale bytes."""
    lens: list
    news: list
    table: np.ndarray
    k: np.ndarray
    v: np.ndarray
    k_scale: np.ndarray
    v_scale: np.ndarray

    @property
    def page(self):
        return self.k.shape[2]

    @property
    def starts(self):
        return np.concatenate([[0], np.cumsum(self.news)])

    @property
    def positions(self):
        """Place of each new token in its sequence."""
        return np.concatenate([n - m + np.arange(m) for n, m in zip(self.lens, self.news)]).astype(np.int64)

    def cache(self):
        return (*(torch.from_numpy(packed(c)).cuda() for c in (self.k, self.v)),
                *(torch.from_numpy(s.copy()).cuda().view(torch.float8_e5m2) for s in (self.k_scale, self.v_scale)))

    def device(self, uniform: bool | None = None):
        """(cache tensors, page_table, lens, cu_q or None) on the GPU."""
        same = len(set(self.news)) <= 1 if uniform is None else uniform
        cu = None if same else torch.from_numpy(self.starts.astype(np.int32)).cuda()
        return self.cache(), torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"), cu


def make_batch(seed, lens, news, heads, dim, page, *, garbage=True, spare=2, size=1.0) -> Batch:
    """A cache whose pages are scattered; unused slots and spare pages hold any codes and scales
    that are infinite, no numbers or negative."""
    rng = np.random.default_rng([seed, heads, dim, page, len(lens)])
    counts = [-(-n // page) for n in lens]
    pages, width = sum(counts) + spare, max(max(counts), 1)
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    used = np.zeros((pages, page), bool)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        used[table[b, np.arange(lens[b]) // page], np.arange(lens[b]) % page] = True
        at += c
    both = []
    for _ in range(2):
        loud = np.exp(rng.standard_normal((heads, 1, dim)) * 0.7) * size
        codes, scales = coded(rng.standard_normal((pages, heads, page, dim)) * loud)
        if garbage:
            keep = used[:, None, :, None]
            codes = np.where(keep, codes, rng.integers(0, 16, codes.shape)).astype(np.uint8)
            scales = np.where(keep, scales, rng.choice([0x7C, 0x7D, 0x7F, 0xFF, 0xFC, 0x9A], scales.shape)).astype(np.uint8)
        both.append((codes, scales))
    return Batch(list(lens), list(news), table, both[0][0], both[1][0], both[0][1], both[1][1])


def normed(x, weight, eps):
    """fp64 [tokens, heads, dim] over its root mean square, times weight."""
    if weight is None:
        return x
    with np.errstate(divide="ignore", invalid="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def rotated(x, positions, turns, axes, interleaved, factor):
    """(fp64 rows turned, |a| + |b| behind each value): positions [tokens] or [tokens, axes]."""
    if not len(turns):
        return x, np.abs(x)
    p = positions[:, None] if positions.ndim == 1 else positions[:, axes]
    p = np.broadcast_to(p, (len(x), len(turns)))
    ph = [[((int(a) * int(t) + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64 for a, t in zip(row, turns)] for row in p]
    th = 2 * math.pi * np.array(ph).reshape(len(x), 1, len(turns))
    c, s, half = np.cos(th) * factor, np.sin(th) * factor, len(turns)
    i = np.arange(half)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out, mag = x.copy(), np.abs(x)
    out[..., i], out[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    mag[..., i] = mag[..., j] = (np.abs(x[..., i]) + np.abs(x[..., j])) * abs(factor)
    return out, mag


def cached(b: Batch, seq: int, head: int, which: str):
    """(fp64 [len, dim] of a sequence's keys or values of one head, the largest that codes of
    such scales can stand for)."""
    codes, scales = (b.k, b.k_scale) if which == "k" else (b.v, b.v_scale)
    n, dim = b.lens[seq], b.k.shape[3]
    ids = b.table[seq, :-(-n // b.page)].astype(np.int64) if n else np.zeros(0, np.int64)
    inside = ((ids >= 0) & (ids < codes.shape[0]))[:, None, None]
    safe = np.clip(ids, 0, codes.shape[0] - 1)
    x = np.where(inside, values(codes[safe, head], scales[safe, head]), 0.0)
    top = np.where(inside, np.repeat(np.nan_to_num(np.abs(E5M2[scales[safe, head]]), posinf=0.0), GROUP, -1), 0.0) * 16
    return x.reshape(-1, dim)[:n], top.reshape(-1, dim)[:n]


def attention(q: np.ndarray, b: Batch, scale: float, window: int = 0):
    """(out, lse, bound, lse_bound): q fp64 [T, heads, dim].

    The bounds on |kernel - out| follow from the kernel's arithmetic.  Scores: codes 0 .. 15, or
    their values, summed in fp32 with the share of the offset taken off, some ten roundings of
    sums of up to |q| 16 s (2^-20 of it); q in fp16 to 2^-31 of its row's largest.  2^x
    to 2^-22.  Weights in fp16: 2^-11 of themselves or 2^-32 of the largest.  Products with v
    exact, summed in fp32 (2^-19 of the magnitudes); out rounded to bf16 (2^-8 of the value)."""
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
        for h in range(heads):
            (k, ktop), (v, _) = cached(b, s, h // group, "k"), cached(b, s, h // group, "v")
            x = np.where(seen, q[rows, h] @ np.nan_to_num(k).T * scale, -np.inf)
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
            mag = np.abs(q[rows, h]) @ ktop.T * abs(scale)
            far = np.abs(q[rows, h]).max(1, keepdims=True, initial=0.0) * ktop.sum(1)[None] * abs(scale) * 2.0 ** -31
            d = np.where(seen, (mag + np.abs(np.nan_to_num(x, neginf=0.0)) + 1.0) * 2.0 ** -20 + far, 0.0)
            av = np.abs(np.nan_to_num(v))
            rel = d + np.max(d, 1, keepdims=True, initial=0.0) + 2.0 ** -11 + 2.0 ** -19
            top = np.max(p, 1, keepdims=True, initial=0.0)
            bound[rows, h] = 2.0 ** -8 * np.abs(np.nan_to_num(o)) + (p * rel) @ av + 2.0 ** -32 * top * (seen.astype(float) @ av) + 1e-30
            lse_bound[rows, h] = 2.0 * np.max(d, 1, initial=0.0) + 2.0 ** -21 * np.abs(np.nan_to_num(lse[rows, h], neginf=0.0)) + 2.0 ** -18
    return out, lse, bound, lse_bound
