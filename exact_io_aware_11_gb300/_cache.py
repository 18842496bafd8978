"""Binding of the rotary and cache entry points of libfa.so: rotary positions,
a paged key/value cache held in 8 bits, and attention over it.

As in _lib.py, every step of the computation runs in the CUDA kernels; this
module checks and marshals tensors and allocates outputs. Calls run on the
tensors' device; outputs and workspaces that a call allocates belong to the
stream it runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from ._lib import _I, _P, FA_OK, SIGNATURES, FaError, lib

_I32, _I64, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}


def _strides(name):
    return [(f"{name}_{a}", _I64) for a in "bhn"]


class RotaryOptions(ctypes.Structure):
    """fa_rotary_options of include/fa.h."""
    _fields_ = [("rotary_dim", _I), ("interleaved", _I), ("dtype", _I), ("factor", _F), ("turns", _P), ("positions", _P),
                ("pos_stride_b", _I64), ("pos_stride_n", _I64), ("offset", _I32),
                *_strides("q"), *_strides("q_out"), *_strides("k"), *_strides("k_out")]


class CacheStruct(ctypes.Structure):
    """fa_cache of include/fa.h."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("num_pages", _I), ("H", _I), ("page_size", _I),
                ("d", _I), ("format", _I)]


class CacheRange(ctypes.Structure):
    """fa_cache_range of include/fa.h."""
    _fields_ = [("page_table", _P), ("table_stride", _I64), ("table_width", _I), ("start", _P), ("count", _P), ("dtype", _I),
                *_strides("x")]


class CacheAttentionOptions(ctypes.Structure):
    """fa_cache_attention_options of include/fa.h."""
    _fields_ = [("page_table", _P), ("table_stride", _I64), ("table_width", _I), ("kv_len", _P), ("q_len", _P),
                ("causal", _I), ("dtype", _I), ("scale", _F), *_strides("q"), *_strides("o")]


_SZ = ctypes.c_size_t
SIGNATURES["fa_rotary_fwd"] = SIGNATURES["fa_rotary_bwd"] = (
    _I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.POINTER(RotaryOptions), _P])
SIGNATURES["fa_cache_write"] = SIGNATURES["fa_cache_read"] = (
    _I, [ctypes.POINTER(CacheStruct), _P, _P, _I, _I, ctypes.POINTER(CacheRange), _P])
SIGNATURES["fa_cache_attention_workspace_bytes"] = (_SZ, [ctypes.POINTER(CacheStruct), _I, _I, _I, _I])
SIGNATURES["fa_cache_attention"] = (_I, [_P, _P, _P, ctypes.POINTER(CacheStruct), _I, _I, _I,
                                         ctypes.POINTER(CacheAttentionOptions), _P, _SZ, _P])

_SAME = contextlib.nullcontext()


def _on(device, stream):
    """Context that makes `device` current and, if one is given, `stream`."""
    if stream is not None:
        return torch.cuda.stream(stream)
    return _SAME if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _check_stream(device, stream):
    if stream is not None and stream.device != device:
        raise ValueError("the stream belongs to another device than the tensors")


def _check_rows(t, what, device=None, dtype=None):
    """A CUDA bf16 or fp16 [B, H, N, d] view with a contiguous d axis."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype not in _DTYPES or t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{what} must be a bf16 or fp16 [B, H, N, d] view with a contiguous last axis")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on another device")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} has another dtype than the call's other tensors")


def _row_strides(t):
    """Element strides (b, h, n), 0 on axes that are never stepped."""
    s, n = t.stride(), t.shape
    out = (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)
    if out == (0, 0, 0) and n[0] * n[1] * n[2] > 1:
        raise ValueError("rows must not overlap")  # three zeros would mean row-major
    return out


def _check_int(t, what, device, dim):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device or t.dim() != dim:
        raise ValueError(f"{what} must be an int32 tensor of {dim} dimension(s) on the tensors' device")


def _check_lengths(t, what, device, B):
    if t is None:
        return None
    _check_int(t, what, device, 1)
    if t.shape[0] != B or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous, one value per sequence")
    return t.data_ptr()


def _check_table(t, device, B):
    _check_int(t, "page_table", device, 2)
    if t.shape[0] != B or t.shape[1] < 1 or t.stride(1) != 1:
        raise ValueError("page_table must be [B, pages per sequence] with a contiguous last axis")
    return t.data_ptr(), t.stride(0) if B > 1 else 0, t.shape[1]


def _like(t):
    """An empty tensor of t's shape that keeps [B, N, H, d] storage where t has it."""
    return torch.empty_like(t)


def _done(rc, where):
    if rc != FA_OK:
        raise FaError(rc, where)


# ------------------------------------------------------------------ rotary positions
class Rotary:
    """Frequencies of rotary positions: what each pair of channels turns per
    position (64-bit fractions of a turn, on the device), the factor on cos
    and sin, and the layout of the pairs. Made by rotary_frequencies, or from
    any angles per position (radians, float64 [rotary_dim / 2])."""

    def __init__(self, angles, factor: float = 1.0, interleaved: bool = False, device="cuda"):
        angles = torch.as_tensor(angles, dtype=torch.float64).cpu()
        if angles.dim() != 1 or angles.numel() < 1 or not bool(torch.isfinite(angles).all()):
            raise ValueError("angles must be a vector of finite numbers")
        if not math.isfinite(factor):
            raise ValueError("factor must be finite")
        # angle / 2 pi modulo 1, times 2^64, in a signed word of the same bits
        turns = [int(round(math.fmod(a / (2 * math.pi), 1.0) * 2.0 ** 64)) & (2 ** 64 - 1) for a in angles.tolist()]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        self.angles, self.factor, self.interleaved = angles, float(factor), bool(interleaved)
        self.rotary_dim = 2 * angles.numel()


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                       interleaved: bool = False, device="cuda") -> Rotary:
    """The frequencies base^(-2i / rotary_dim) of pair i, scaled for contexts
    `factor` times as long as the trained one:
      None      as they are;
      "linear"  all divided by factor (position interpolation);
      "ntk"     the base times factor^(rotary_dim / (rotary_dim - 2)), which leaves the
                fastest pair and divides the slowest by factor;
      "yarn"    pairs that turn more than beta_fast times over original_length as they
                are, those that turn less than beta_slow times divided by factor, a linear
                ramp over the pairs between; cos and sin times 0.1 ln(factor) + 1."""
    r = int(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (math.isfinite(base) and base > 0) or not (math.isfinite(factor) and factor > 0):
        raise ValueError("base and factor must be finite and positive")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if scaling == "ntk":
        if r == 2:
            raise ValueError("ntk scaling needs more than one pair")
        base = base * factor ** (r / (r - 2))
    i = torch.arange(r // 2, dtype=torch.float64)
    w = base ** (-2.0 * i / r)
    attention = 1.0
    if scaling == "linear":
        w = w / factor
    elif scaling == "yarn":
        if original_length is None or original_length < 1:
            raise ValueError("yarn scaling needs original_length")
        if not (beta_fast > 0 and beta_slow > 0) or base <= 1:
            raise ValueError("yarn scaling needs positive betas and a base above 1")

        def pair_of(turns):  # the (real) pair that turns so often over original_length
            return r * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        low, high = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), r - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        w = w / factor * ramp + w * (1 - ramp)
        attention = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return Rotary(w, attention, interleaved, device)


def _rotary(name, q, rotary, k, positions, offset, out, k_out, stream):
    _check_rows(q, "q")
    dev = q.device
    B, Hq, N, d = q.shape
    if not isinstance(rotary, Rotary) or rotary.turns.device != dev:
        raise ValueError("rotary must be a Rotary on the tensors' device")
    if k is not None:
        _check_rows(k, "k", dev, q.dtype)
        if k.shape[0] != B or k.shape[2:] != q.shape[2:]:
            raise ValueError("k must be [B, heads, N, d] with q's B, N and d")
    elif k_out is not None:
        raise ValueError("k_out without k")
    ps = (None, 0, 0)
    if positions is not None:
        if offset:
            raise ValueError("give positions or an offset, not both")
        if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
            raise ValueError("positions must be int32 [N] or [B, N]")
        _check_int(positions, "positions", dev, positions.dim())
        if positions.shape[-1] != N or (positions.dim() == 2 and positions.shape[0] != B):
            raise ValueError("positions must be int32 [N] or [B, N]")
        ps = (positions.data_ptr(), positions.stride(0) if positions.dim() == 2 else 0, positions.stride(-1))
    if not -2 ** 31 <= int(offset) < 2 ** 31:
        raise ValueError("offset must fit in 32 bits")
    _check_stream(dev, stream)
    with _on(dev, stream):
        y = _like(q) if out is None else out
        z = None if k is None else _like(k) if k_out is None else k_out
        if out is not None:
            _check_rows(out, "out", dev, q.dtype)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        if k_out is not None:
            _check_rows(k_out, "k_out", dev, q.dtype)
            if k_out.shape != k.shape:
                raise ValueError("k_out must have k's shape")
        none = (0, 0, 0)
        opt = RotaryOptions(rotary.rotary_dim, int(rotary.interleaved), _DTYPES[q.dtype], rotary.factor,
                            rotary.turns.data_ptr(), *ps, int(offset), *_row_strides(q), *_row_strides(y),
                            *(none if k is None else _row_strides(k)), *(none if k is None else _row_strides(z)))
        _done(getattr(lib(), name)(q.data_ptr(), y.data_ptr(), None if k is None else k.data_ptr(),
                                   None if k is None else z.data_ptr(), B, Hq, 0 if k is None else k.shape[1], N, d, opt,
                                   torch.cuda.current_stream(dev).cuda_stream), name)
    return y if k is None else (y, z)


def rotary_forward(q, rotary: Rotary, k=None, positions=None, offset: int = 0, out=None, k_out=None, stream=None):
    """q [B, H, N, d] with the first rotary.rotary_dim channels of each row turned to
    its position (fa_rotary_fwd); with k [B, Hk, N, d], (q, k) in one launch.
    positions: int32 [N] or [B, N] on the device, or None for offset + n.
    out=q (k_out=k) rotates in place."""
    return _rotary("fa_rotary_fwd", q, rotary, k, positions, offset, out, k_out, stream)


def rotary_backward(dq, rotary: Rotary, dk=None, positions=None, offset: int = 0, out=None, k_out=None, stream=None):
    """Gradients with respect to rotary_forward's inputs from those of its outputs
    (fa_rotary_bwd), with the same rotary and positions: dq, or (dq, dk)."""
    return _rotary("fa_rotary_bwd", dq, rotary, dk, positions, offset, out, k_out, stream)


# ------------------------------------------------------------------ the cache
class KVCache:
    """The page pool of one layer (fa_cache): codes k, v [num_pages, H, page_size, d]
    (torch.float8_e4m3fn or torch.int8) and fp32 scales k_scale, v_scale [num_pages, H],
    one for each page and head; a row stands for code * scale. Which pages a sequence has is
    the caller's page table, int32 [B, pages per sequence]. KVCache.empty makes a pool."""

    def __init__(self, k, v, k_scale, v_scale):
        for t in (k, v):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _FORMATS or t.dim() != 4 or not t.is_contiguous():
                raise ValueError("k and v must be contiguous float8_e4m3fn or int8 CUDA tensors [num_pages, H, page_size, d]")
        if v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("k and v must have the same shape, dtype and device")
        P, H, page, d = k.shape
        for t in (k_scale, v_scale):
            if (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.device != k.device
                    or tuple(t.shape) != (P, H) or not t.is_contiguous()):
                raise ValueError("k_scale and v_scale must be contiguous float32 [num_pages, H] on the codes' device")
        if page not in (16, 32, 64, 128) or d not in (64, 128):
            raise ValueError("page_size must be 16, 32, 64 or 128 and d 64 or 128")
        self._tensors = (k, v, k_scale, v_scale)
        self._struct = CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), P, H, page, d,
                                   _FORMATS[k.dtype])

    @classmethod
    def empty(cls, num_pages: int, heads: int, head_dim: int, page_size: int = 64, dtype=torch.float8_e4m3fn, device="cuda"):
        """A pool of zeros."""
        codes = [torch.zeros((num_pages, heads, page_size, head_dim), dtype=torch.int8, device=device).view(dtype) for _ in "kv"]
        return cls(*codes, *(torch.zeros((num_pages, heads), dtype=torch.float32, device=device) for _ in "kv"))

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])
    page_size = property(lambda self: self._struct.page_size)
    heads = property(lambda self: self._struct.H)
    head_dim = property(lambda self: self._struct.d)


def _check_cache(cache):
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    return cache.k.device


def _cache_rows(name, cache, k, v, page_table, start, count, stream):
    dev = cache.k.device
    B, H, N, d = k.shape
    if v.shape != k.shape or H != cache.heads or d != cache.head_dim:
        raise ValueError("k and v must be [B, H, N, d] with the cache's H and d")
    if _row_strides(k) != _row_strides(v):
        raise ValueError("k and v must share strides")
    rng = CacheRange(*_check_table(page_table, dev, B), _check_lengths(start, "start", dev, B),
                     _check_lengths(count, "count", dev, B), _DTYPES[k.dtype], *_row_strides(k))
    _done(getattr(lib(), name)(cache._struct, k.data_ptr(), v.data_ptr(), B, N, rng,
                               torch.cuda.current_stream(dev).cuda_stream), name)


def cache_write(cache: KVCache, k, v, page_table, start, count=None, stream=None) -> None:
    """Quantises rows n < count[b] of k, v [B, H, N, d] into the cache at tokens
    start[b] + n (fa_cache_write). start, count: int32 [B]; start=None means 0,
    count=None all N rows. Where a page is shared by the old and the new tokens of a
    sequence, its older rows move to the page's new scale if that grew. Two
    sequences of one call must not write the same page."""
    dev = _check_cache(cache)
    _check_rows(k, "k", dev)
    _check_rows(v, "v", dev, k.dtype)
    _check_stream(dev, stream)
    with _on(dev, stream):
        _cache_rows("fa_cache_write", cache, k, v, page_table, start, count, stream)


def cache_read(cache: KVCache, page_table, count, N: int, start=None, dtype=torch.bfloat16, k_out=None, v_out=None,
               stream=None):
    """k, v [B, H, N, d] of tokens start[b] + n, n < count[b], of the cache, in dtype
    (fa_cache_read); rows n >= count[b] are zeros."""
    dev = _check_cache(cache)
    _check_int(page_table, "page_table", dev, 2)
    if int(N) < 1:
        raise ValueError("N must be at least 1")
    if (k_out is None) != (v_out is None):
        raise ValueError("give both k_out and v_out, or neither")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be bf16 or fp16")
    _check_stream(dev, stream)
    with _on(dev, stream):
        shape = (page_table.shape[0], cache.heads, int(N), cache.head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=dev) if t is None else t for t in (k_out, v_out))
        for t in (k, v):
            _check_rows(t, "k_out, v_out", dev, dtype)
            if tuple(t.shape) != shape:
                raise ValueError("k_out and v_out must be [B, H, N, d]")
        _cache_rows("fa_cache_read", cache, k, v, page_table, start, count, stream)
    return k, v


def cache_attention_workspace_bytes(cache: KVCache, B: int, heads: int, N: int, pages: int) -> int:
    """Workspace bytes with which cache_attention spreads sequences over every SM, for q
    [B, heads, N, d] and a page table of `pages` columns (0: none needed)."""
    dev = _check_cache(cache)
    with _on(dev, None):
        return int(lib().fa_cache_attention_workspace_bytes(cache._struct, B, heads, N, pages))


def cache_attention(q, cache: KVCache, page_table, kv_len, q_len=None, causal: bool = True, scale: float | None = None,
                    out=None, lse=None, workspace=None, stream=None, split: bool = True):
    """O, LSE of q [B, H, N, d] over the cache's tokens j < kv_len[b] (fa_cache_attention);
    H is a multiple of the cache's heads. Causal: row i < q_len[b] (default N) sits at
    token kv_len[b] - q_len[b] + i, so the newest tokens are written before the call. Rows
    that see no token, and rows i >= q_len[b], get O = 0 and LSE = -inf. `workspace`:
    uint8 of cache_attention_workspace_bytes(...) bytes, kept by the caller, allocated
    here if None; split=False does without."""
    dev = _check_cache(cache)
    _check_rows(q, "q", dev)
    B, H, N, d = q.shape
    if d != cache.head_dim or H % cache.heads:
        raise ValueError("q must have the cache's d and a multiple of its heads")
    _check_stream(dev, stream)
    if kv_len is None:
        raise ValueError("kv_len is needed")
    table, table_stride, pages = _check_table(page_table, dev, B)
    with _on(dev, stream):
        o = _like(q) if out is None else out
        if out is not None:
            _check_rows(out, "out", dev, q.dtype)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        if lse is None:
            l = torch.empty((B, H, N), dtype=torch.float32, device=dev)
        else:
            l = lse
            if l.dtype != torch.float32 or l.device != dev or tuple(l.shape) != (B, H, N) or not l.is_contiguous():
                raise ValueError("lse must be contiguous float32 [B, H, N]")
        ws = workspace
        if ws is None and split:
            need = lib().fa_cache_attention_workspace_bytes(cache._struct, B, H, N, pages)
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        elif ws is not None and (not ws.is_cuda or ws.device != dev or not ws.is_contiguous()):
            raise ValueError("workspace must be a contiguous CUDA tensor on the tensors' device")
        n = ws.numel() * ws.element_size() if ws is not None else 0
        opt = CacheAttentionOptions(table, table_stride, pages, _check_lengths(kv_len, "kv_len", dev, B),
                                    _check_lengths(q_len, "q_len", dev, B), int(bool(causal)), _DTYPES[q.dtype],
                                    d ** -0.5 if scale is None else float(scale), *_row_strides(q), *_row_strides(o))
        _done(lib().fa_cache_attention(q.data_ptr(), o.data_ptr(), l.data_ptr(), cache._struct, B, H, N, opt,
                                       ws.data_ptr() if n else None, n, torch.cuda.current_stream(dev).cuda_stream),
              "fa_cache_attention")
    return o, l
