"""What a decode step does between the linear layers: norms of the heads, rotary positions
and the write into an 8-bit or 4-bit key-value cache, attention over that cache, and sampling.

Same rules as the linear layer's binding (``_abi``): tensors on the GPU with the
dtypes include/lowbit.h documents, argument marshalling only, the current CUDA
stream, and ``LowbitError`` for a non-zero status.

The cache is four tensors: ``k`` and ``v`` [pages, kv_heads, page, head_dim] in
``torch.float8_e4m3fn`` (``uint8`` bit patterns are taken too) and ``k_exp``, ``v_exp``
[pages, kv_heads] int8: value = code * 2**exp, one exponent for each page of tokens and
head (``empty_cache`` makes them).  In 4 bits (``empty_cache(..., bits=4)``) they are ``k``
and ``v`` [pages, kv_heads, page, head_dim / 2] uint8, two codes a byte, and a scale for each
32 values of a token's head, [pages, kv_heads, page, head_dim / 32] ``torch.float8_e5m2``, in
the place of the exponents: value = (code - 8) * scale.  Every function takes either kind.
``page_table`` [batch, width] int32 names each
sequence's pages in order, ``lens`` [batch] int32 its length with its new tokens.
The new tokens of all sequences stand one after another; ``cu_q`` [batch + 1] int32 says
where each sequence's begin (None: the same number of tokens each).
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import struct

import torch

from . import _abi
from . import build as _build

_hot = None


def _load():
    """The extension module that makes the accepted calls (csrc/binding.cpp)."""
    global _hot
    if _hot is None:
        lib = _abi.abi()
        path = _build.binding()
        if not path.exists():
            raise ImportError(f"_lowbit_torch is not built ({path} missing); run bit_groupwise_weight_gb300.build.build()")
        spec = importlib.util.spec_from_file_location("_lowbit_torch", str(path))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.lowbit_kv_append_ex, lib.lowbit_kv_append4, lib.lowbit_attention, lib.lowbit_attention4,
            lib.lowbit_attention_workspace, lib.lowbit_attention4_workspace, lib.lowbit_cache_values, lib.lowbit_cache4_values,
            lib.lowbit_sample)))
        _hot = module
    return _hot


# What follows describes a call in Python: how one that the extension did not accept is
# explained.  The C ABI's descriptors, packed:
def _packer(layout: str, of: str):
    pack = struct.Struct(layout).pack

    def packed(*values):
        try:
            return pack(*values)
        except (struct.error, OverflowError) as e:      # not a number, or past 32 bits
            raise ValueError(f"a number among {of} is not one or does not fit: {e}") from None
    return packed


_CACHE = _packer("@PPPPqqiiii", "the cache's sizes")                       # lowbit_cache
_CACHE4 = _packer("@PPPPqqqqiiii", "the cache's sizes")                    # lowbit_cache4
_PROLOGUE = _packer("@PPPPqfii4x", "the axes, the positions' stride and eps")  # lowbit_kv_prologue
_SEQUENCES = _packer("@PPPqiiii", "the sequences' sizes and max_q")        # lowbit_sequences
_KV_APPEND = _packer("@PPPPqqqqqqqqPfiii", "the sizes and factor")
_ATTENTION = _packer("@PPPqqqqqPNfii4x", "the sizes, scale and window")
_SAMPLE = _packer("@PPPPPPPPqfffiiii4x", "the sizes, temperature, top_p, min_p and top_k")

_BF16, _F32, _I32, _I8, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.int64, torch.uint8
_CODES = (torch.float8_e4m3fn, _U8)
_SCALES = (torch.float8_e5m2, _U8)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else _abi._stream


def _call(fn, name: str, dev: int, *args) -> None:
    if torch.cuda.current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _abi._check(status, name)


def _refuse(t, name: str, dtypes, dev: int, shape: tuple):
    """Raises the error that explains why a tensor did not pass (None in the shape: any size)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"all tensors must be on one device, got cuda:{dev} and {t.device}")
    if t.dim() != len(shape) or any(want is not None and got != want for got, want in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple('*' if n is None else n for n in shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous" + (" in its last dimension" if len(shape) > 1 else ""))


def _vector(t, name: str, dtype, dev: int, n: int) -> int:
    """Address of a contiguous tensor of one dimension."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == (n,) and t.is_contiguous()):
        _refuse(t, name, (dtype,), dev, (n,))
    return t.data_ptr()


def _first(q, name: str, ndim: int) -> int:
    """Device of the tensor that the others have to be with."""
    if not isinstance(q, torch.Tensor) or q.dim() != ndim or not q.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of {ndim} dimensions")
    return q.get_device()


def _rows(t, name: str, dev: int, T: int, H: int, D: int):
    """(address, token stride, head stride) of bf16 [T, H, D], contiguous in the last dimension."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == dev and t.shape == (T, H, D):
        token, head, one = t.stride()
        if one == 1:
            return t.data_ptr(), token, head
    _refuse(t, name, (_BF16,), dev, (T, H, D))


class _Cache:
    """A cache's descriptor, and the library's functions that take it."""

    def __init__(self, packed, kv_heads: int, bits: int):
        self.packed, self.kv_heads, self.bits = packed, kv_heads, bits

    def fn(self, what: str):
        names = {"append": ("lowbit_kv_append_ex", "lowbit_kv_append4"), "attention": ("lowbit_attention", "lowbit_attention4"),
                 "workspace": ("lowbit_attention_workspace", "lowbit_attention4_workspace"),
                 "values": ("lowbit_cache_values", "lowbit_cache4_values")}
        return getattr(_abi.abi(), names[what][self.bits == 4])


def _pair_of(k, v, names, dtypes, dev: int):
    """Strides of two tensors [pages, kv_heads, page, n] with the same strides, each head's page contiguous."""
    if not (isinstance(k, torch.Tensor) and k.dtype in dtypes and k.get_device() == dev and k.dim() == 4):
        _refuse(k, names[0], dtypes, dev, (None,) * 4)
    if not (isinstance(v, torch.Tensor) and v.dtype in dtypes and v.get_device() == dev and v.shape == k.shape):
        _refuse(v, names[1], dtypes, dev, tuple(k.shape))
    strides = k.stride()
    if strides != v.stride() or (strides[2] != k.shape[3] or strides[3] != 1) and k.numel():
        raise ValueError(f"{names[0]} and {names[1]} must have the same strides, each head's page contiguous")
    return strides


def _cache_of(k, v, k_exp, v_exp, dev: int, dim: int) -> _Cache:
    if isinstance(k_exp, torch.Tensor) and k_exp.dim() == 4:                  # scales: the 4-bit kind
        strides = _pair_of(k, v, ("k_cache", "v_cache"), (_U8,), dev)
        pages, heads, page, half = k.shape
        if 2 * half != dim:
            raise ValueError(f"q has head_dim {dim}, the cache {2 * half}")
        apart = _pair_of(k_exp, v_exp, ("k_exp", "v_exp"), _SCALES, dev)
        if dim % 32 or tuple(k_exp.shape) != (pages, heads, page, dim // 32):
            _refuse(k_exp, "k_exp", _SCALES, dev, (pages, heads, page, dim // 32))
        return _Cache(_CACHE4(k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), strides[0], strides[1], apart[0],
                              apart[1], pages, heads, dim, page), heads, 4)
    strides = _pair_of(k, v, ("k_cache", "v_cache"), _CODES, dev)
    pages, heads, page, d = k.shape
    if d != dim:
        raise ValueError(f"q has head_dim {dim}, the cache {d}")
    for t, name in ((k_exp, "k_exp"), (v_exp, "v_exp")):
        if not (isinstance(t, torch.Tensor) and t.dtype is _I8 and t.get_device() == dev and t.shape == (pages, heads)
                and t.is_contiguous()):
            _refuse(t, name, (_I8,), dev, (pages, heads))
    return _Cache(_CACHE(k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), strides[0], strides[1], pages, heads, d,
                         page), heads, 8)


def _prologue_of(q_norm, k_norm, eps, positions, axes, dev: int, tokens: int, dim: int, pairs: int):
    """lowbit_kv_prologue."""
    at, dtype = [0, 0], None
    for i, (w, name) in enumerate(((q_norm, "q_norm"), (k_norm, "k_norm"))):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor) or w.dtype not in _abi._W_DTYPES:
            raise ValueError(f"{name} must be a float32, bfloat16 or float16 CUDA tensor")
        if dtype not in (None, w.dtype):
            raise ValueError(f"q_norm and k_norm must have one dtype, got {dtype} and {w.dtype}")
        dtype = w.dtype
        at[i] = _vector(w, name, dtype, dev, dim)
    where = token = count = axes_at = 0
    if positions is None:
        if axes is not None:
            raise ValueError("axes say which column of positions each pair turns by: they need positions")
    else:
        if not (isinstance(positions, torch.Tensor) and positions.dtype is _I32 and positions.get_device() == dev
                and positions.dim() in (1, 2) and positions.shape[0] == tokens):
            _refuse(positions, "positions", (_I32,), dev, (tokens,) + (None,) * (isinstance(positions, torch.Tensor) and positions.dim() > 1))
        where, token, count = positions.data_ptr(), positions.stride(0), 1 if positions.dim() == 1 else positions.shape[1]
        if not 1 <= count <= 255:
            raise ValueError(f"positions must have 1 to 255 axes, got {count}")
        if count > 1 and positions.stride(1) != 1:
            _refuse(positions, "positions", (_I32,), dev, (tokens, None))
        if axes is not None:
            axes_at = _vector(axes, "axes", _U8, dev, pairs)
        elif count > 1:
            raise ValueError("positions of several axes need axes: the one that each pair turns by")
    return _PROLOGUE(*at, where, axes_at, token, eps, count, 0 if dtype is None else _abi._W_DTYPES[dtype])


def _sequences_of(page_table, lens, cu_q, max_q, tokens: int, dev: int):
    if not (isinstance(page_table, torch.Tensor) and page_table.dtype is _I32 and page_table.get_device() == dev
            and page_table.dim() == 2):
        _refuse(page_table, "page_table", (_I32,), dev, (None, None))
    batch, width = page_table.shape
    apart, one = page_table.stride()
    if (one != 1 and width > 1) or (apart < width and batch > 1):
        raise ValueError("the rows of page_table must be contiguous and apart")
    lens_at = _vector(lens, "lens", _I32, dev, batch)
    if cu_q is None:
        if batch and tokens % batch:
            raise ValueError(f"without cu_q, {batch} sequences must have the same number of new tokens, got {tokens} in all")
        cu_at, max_q = 0, tokens // batch if batch else 0
    else:
        cu_at, max_q = _vector(cu_q, "cu_q", _I32, dev, batch + 1), tokens if max_q is None else max_q
    return _SEQUENCES(page_table.data_ptr(), lens_at, cu_at, max(apart, width), width, batch, tokens, max_q)


def empty_cache(pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda", bits: int = 8):
    """(k, v, k_exp, v_exp) of a cache of ``pages`` pages of ``page`` tokens, zeroed; with ``bits=4``
    (k, v, k_scale, v_scale), half the size: 4.25 bits a value."""
    if bits not in (4, 8):
        raise ValueError(f"bits must be 4 or 8, got {bits}")
    if bits == 4:
        if head_dim not in (64, 128):
            raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
        k, v = (torch.zeros((pages, kv_heads, page, head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2))
        k_scale, v_scale = (torch.zeros((pages, kv_heads, page, head_dim // 32), dtype=torch.uint8, device=device)
                            .view(torch.float8_e5m2) for _ in range(2))
        return k, v, k_scale, v_scale
    k, v = (torch.zeros((pages, kv_heads, page, head_dim), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
            for _ in range(2))
    k_exp, v_exp = (torch.zeros((pages, kv_heads), dtype=torch.int8, device=device) for _ in range(2))
    return k, v, k_exp, v_exp


def cache_values(k_cache, v_cache, k_exp, v_exp, out=(None, None)):
    """(k, v): the values that a cache holds, bf16 [pages, kv_heads, page, head_dim] (or writes the
    two tensors ``out``).  Exact: a value of either kind of cache is a bf16 number."""
    k_out, v_out = out
    done = (_hot or _load()).cache_values(k_cache, v_cache, k_exp, v_exp, k_out, v_out)
    if done is not None:
        return done if done.__class__ is not int else _abi._check(done, "lowbit_cache_values")
    dev = _first(k_cache, "k_cache", 4)
    pages, heads, page, n = k_cache.shape
    dim = 2 * n if isinstance(k_exp, torch.Tensor) and k_exp.dim() == 4 else n
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp, dev, dim)
    shape, outs = (pages, heads, page, dim), []
    for t, name in ((k_out, "out[0]"), (v_out, "out[1]")):
        if t is None:
            t = torch.empty(shape, dtype=_BF16, device=k_cache.device)
        elif not (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == dev and t.shape == shape and t.is_contiguous()):
            _refuse(t, name, (_BF16,), dev, shape)
        outs.append(t)
    _call(cache.fn("values"), "lowbit_cache_values", dev, cache.packed, outs[0].data_ptr(), outs[1].data_ptr())
    return tuple(outs)


def rotary_turns(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                 original_length: int = 8192, low: float = 1.0, high: float = 4.0, device=None) -> torch.Tensor:
    """Frequencies of a rotation over ``dim`` values, as ``kv_append`` takes them: int64
    [dim / 2], turns per position times 2**64.  Pair j turns by base**(-2j/dim) radians a
    position.  ``scaling`` stretches them by ``factor`` for longer contexts than the
    ``original_length`` a model was trained on:

      "linear"      every frequency divided by factor;
      "base"        the base raised so that the slowest pair slows by factor and the
                    fastest not at all;
      "wavelength"  pairs that turn more than ``high`` times over the original length
                    keep their frequency, those that turn less than ``low`` times are
                    divided by factor, and those between are blended in proportion.
    """
    if dim < 0 or dim % 2:
        raise ValueError(f"dim must be even and not negative, got {dim}")
    if not base > 1 or not factor >= 1 or not original_length > 0 or not high > low:
        raise ValueError("base must be above 1, factor at least 1, original_length positive and high above low")
    if scaling not in (None, "linear", "base", "wavelength"):
        raise ValueError(f'scaling must be None, "linear", "base" or "wavelength", got {scaling!r}')
    if scaling == "base" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    turns = []
    for j in range(dim // 2):
        f = base ** (-2.0 * j / dim) / (2.0 * math.pi)            # turns a position
        if scaling == "linear":
            f /= factor
        elif scaling == "wavelength":
            keep = min(max((f * original_length - low) / (high - low), 0.0), 1.0)
            f = f * keep + f / factor * (1.0 - keep)
        turns.append(int(round(f * 2.0 ** 64)))
    return torch.tensor(turns, dtype=torch.int64, device=device)


def kv_append(q, k, v, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q=None, max_q: int | None = None, turns=None,
              interleaved: bool = False, factor: float = 1.0, out=None, *, q_norm=None, k_norm=None, eps: float = 1e-6,
              positions=None, axes=None) -> torch.Tensor:
    """Rotate q and k to their positions and write k and v into the cache; returns q
    rotated, bf16 [tokens, heads, head_dim] (or writes ``out``, which may be q).

    q [tokens, heads, head_dim], k, v [tokens, kv_heads, head_dim] bf16, contiguous in
    the last dimension (slices of one qkv projection's output do).  ``turns``: from
    ``rotary_turns``, over the head's first 2 * len(turns) values (None: no rotation);
    ``interleaved`` pairs neighbours, otherwise the halves; ``factor`` multiplies the
    rotated part.  ``max_q``: the largest number of new tokens of a sequence (with cu_q;
    None: no bound known).

    Before the rotation, in the same pass: ``q_norm``, ``k_norm`` (bf16, fp16 or fp32 [head_dim],
    either or both), weights by which each head's q or k is multiplied after division by its root
    mean square, sqrt(mean(x * x) + ``eps``).  ``positions`` (int32 [tokens]) are what tokens turn
    by in place of their places in the sequence; with several axes, as time, height and width of
    an image's patches, [tokens, n], and ``axes`` (uint8 [len(turns)]) is the column that each pair
    turns by.  Where a token is written follows from lens all the same.
    """
    if q_norm is None and k_norm is None and positions is None and axes is None:
        done = (_hot or _load()).kv_append(q, k, v, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q, max_q, turns, interleaved,
                                           factor, out)
    else:
        done = (_hot or _load()).kv_append(q, k, v, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q, max_q, turns, interleaved,
                                           factor, out, q_norm, k_norm, eps, positions, axes)
    if done is not None:
        return done if done.__class__ is not int else _abi._check(done, "lowbit_kv_append")
    dev = _first(q, "q", 3)
    T, heads, dim = q.shape
    q_at, qt, qh = _rows(q, "q", dev, T, heads, dim)
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp, dev, dim)
    k_at, kt, kh = _rows(k, "k", dev, T, cache.kv_heads, dim)
    v_at, vt, vh = _rows(v, "v", dev, T, cache.kv_heads, dim)
    turns_at = pairs = 0
    if turns is not None:
        pairs = turns.numel()
        turns_at = _vector(turns, "turns", _I64, dev, pairs)
    seqs = _sequences_of(page_table, lens, cu_q, max_q, T, dev)
    before = _prologue_of(q_norm, k_norm, eps, positions, axes, dev, T, dim, pairs)
    if out is None:
        out = torch.empty_like(q)
    out_at, ot, oh = _rows(out, "out", dev, T, heads, dim)
    args = _KV_APPEND(q_at, k_at, v_at, out_at, qt, qh, kt, kh, vt, vh, ot, oh, turns_at, factor, heads, 2 * pairs,
                      bool(interleaved))
    _call(cache.fn("append"), "lowbit_kv_append", dev, args, before, cache.packed, seqs)
    return out


def attention(q, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q=None, max_q: int | None = None,
              scale: float | None = None, window: int = 0, out=None, lse=None, workspace=None) -> torch.Tensor:
    """Softmax attention of the new tokens' queries over the cache, each over the keys up
    to its own position (the last ``window`` of them if window > 0); returns bf16
    [tokens, heads, head_dim] (or writes ``out``).

    q as ``kv_append`` returns it.  ``scale``: of the scores (None: head_dim ** -0.5).
    ``lse``: fp32 [tokens, heads], receives the scores' log-sum-exp.  ``workspace``: a uint8
    tensor of ``attention_workspace`` bytes to use again from call to call on one stream.
    """
    done = (_hot or _load()).attention(q, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q, max_q, scale, window, out, lse,
                                       workspace)
    if done is not None:
        return done if done.__class__ is not int else _abi._check(done, "lowbit_attention")
    dev = _first(q, "q", 3)
    T, heads, dim = q.shape
    q_at, qt, qh = _rows(q, "q", dev, T, heads, dim)
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp, dev, dim)
    seqs = _sequences_of(page_table, lens, cu_q, max_q, T, dev)
    if out is None:
        out = torch.empty_like(q)
    out_at, ot, oh = _rows(out, "out", dev, T, heads, dim)
    lse_at = lse_token = 0
    if lse is not None:
        if not (isinstance(lse, torch.Tensor) and lse.dtype is _F32 and lse.get_device() == dev and lse.shape == (T, heads)):
            _refuse(lse, "lse", (_F32,), dev, (T, heads))
        lse_token, one = lse.stride()
        if one != 1 and heads > 1:
            _refuse(lse, "lse", (_F32,), dev, (T, heads))
        lse_at = lse.data_ptr()
    if workspace is None:
        workspace = torch.empty(cache.fn("workspace")(heads, cache.packed, seqs), dtype=_U8, device=q.device)
    n = workspace.numel()
    args = _ATTENTION(q_at, out_at, lse_at, qt, qh, ot, oh, lse_token, _vector(workspace, "workspace", _U8, dev, n), n,
                      dim ** -0.5 if scale is None else scale, heads, window)
    _call(cache.fn("attention"), "lowbit_attention", dev, args, cache.packed, seqs)
    return out


def attention_workspace(q, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q=None, max_q: int | None = None) -> int:
    """Bytes of workspace that ``attention`` needs for these tensors."""
    dev = _first(q, "q", 3)
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp, dev, q.shape[2])
    seqs = _sequences_of(page_table, lens, cu_q, max_q, q.shape[0], dev)
    return int(cache.fn("workspace")(q.shape[1], cache.packed, seqs))


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, logprob=None) -> torch.Tensor:
    """One token for each row of logits; returns int64 [rows] (or writes ``out``).

    logits bf16, fp16 or fp32 [rows, vocab], contiguous in the last dimension; u fp32
    [rows] uniform in [0, 1).  ``temperature`` (<= 0: the largest logit), ``top_k`` (0: all),
    ``top_p``, ``min_p``: numbers, or tensors [rows] (fp32; top_k int32).  Kept are the tokens
    whose weight is at least min_p of the likeliest's, of these the top_k likeliest, of these
    the fewest that hold top_p of the mass.  ``logprob``: fp32 [rows], receives the token's
    log-probability among the kept.
    """
    done = (_hot or _load()).sample(logits, u, temperature, top_k, top_p, min_p, out, logprob)
    if done is not None:
        return done if done.__class__ is not int else _abi._check(done, "lowbit_sample")
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _abi._W_DTYPES:
        raise ValueError("logits must be a float32, bfloat16 or float16 CUDA tensor")
    dev = _first(logits, "logits", 2)
    B, V = logits.shape
    row, one = logits.stride()
    if one != 1 and V > 1:
        _refuse(logits, "logits", (logits.dtype,), dev, (None, None))
    u_at = _vector(u, "u", _F32, dev, B)
    t_at = p_at = m_at = k_at = 0                         # per row, or one number for all
    if isinstance(temperature, torch.Tensor):
        t_at, temperature = _vector(temperature, "temperature", _F32, dev, B), 1.0
    if isinstance(top_p, torch.Tensor):
        p_at, top_p = _vector(top_p, "top_p", _F32, dev, B), 1.0
    if isinstance(min_p, torch.Tensor):
        m_at, min_p = _vector(min_p, "min_p", _F32, dev, B), 0.0
    if isinstance(top_k, torch.Tensor):
        k_at, top_k = _vector(top_k, "top_k", _I32, dev, B), 0
    if out is None:
        out = torch.empty_like(u, dtype=_I64)
    args = _SAMPLE(logits.data_ptr(), u_at, t_at, p_at, m_at, k_at, _vector(out, "out", _I64, dev, B),
                   0 if logprob is None else _vector(logprob, "logprob", _F32, dev, B), row, temperature, top_p, min_p,
                   top_k, B, V, _abi._W_DTYPES[logits.dtype])
    _call(_abi.abi().lowbit_sample, "lowbit_sample", dev, args)
    return out
