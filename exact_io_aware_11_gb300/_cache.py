"""Binding of the rotary and cache entry points of libfa.so: rotary positions,
a paged key/value cache held in 8 bits, and attention over it.

As in _lib.py, every step of the computation runs in the CUDA kernels; this
module checks and marshals tensors and allocates outputs. Calls run on the
tensors' device; outputs and workspaces that a call allocates belong to the
stream it runs on.
"""
from __future__ import annotations

import ctypes
import math
import struct

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

SIGNATURES["fa_cache_attention_shared_workspace_bytes"] = (_SZ, [ctypes.POINTER(CacheStruct), _I, _I, _I, _I, _I])
SIGNATURES["fa_cache_attention_shared"] = (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _I, _P, _SZ, _P])  # structs as bytes

# These calls are made once per layer and token: the checks below read each attribute once,
# and the stream comes from the binding that torch.cuda.current_stream wraps (0.1 us against 2), as does
# the device (whose tensors the caller has, so that CUDA is up).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_INT32, _FLOAT32 = torch.int32, torch.float32
_Tensor = torch.Tensor


def _on(call, device, stream, *args):
    """call(*args) with `device` current and, if one is given, `stream`."""
    if stream is not None:
        if stream.device != device:
            raise ValueError("the stream belongs to another device than the tensors")
        with torch.cuda.stream(stream):
            return call(*args)
    if device.index == _raw_device():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _rows(t, what, device=None, dtype=None):
    """Checks a CUDA bf16 or fp16 [B, H, N, d] view with a contiguous d axis; its shape and
    element strides (b, h, n), 0 on axes that are never stepped."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    n, s, dt = t.shape, t.stride(), t.dtype
    if dt not in _DTYPES or len(n) != 4 or s[3] != 1:
        raise ValueError(f"{what} must be a bf16 or fp16 [B, H, N, d] view with a contiguous last axis")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on another device")
    if dtype is not None and dt != dtype:
        raise ValueError(f"{what} has another dtype than the call's other tensors")
    sb, sh, sn = s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0
    if not (sb or sh or sn) and n[0] * n[1] * n[2] > 1:
        raise ValueError("rows must not overlap")  # three zeros would mean row-major
    return n, (sb, sh, sn)


def _check_int(t, what, device, dim):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device or t.dim() != dim:
        raise ValueError(f"{what} must be an int32 tensor of {dim} dimension(s) on the tensors' device")


_OPTIONS = struct.Struct("@PqiPPiifqqqqqq")  # CacheAttentionOptions (packed in a quarter of the constructor's time)
assert _OPTIONS.size == ctypes.sizeof(CacheAttentionOptions)


def _ints(t, what, index, n):
    """The address of a contiguous int32 vector of n values (None: any) on device `index`."""
    if not isinstance(t, _Tensor) or t.dtype is not _INT32 or t.get_device() != index or t.dim() != 1:
        raise ValueError(f"{what} must be an int32 vector on the tensors' device")
    if not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{what} must be contiguous and have {n} values")
    return t.data_ptr()


def _matrix(t, what, index):
    """The address of an int32 [rows, columns] tensor with a contiguous last axis, its row stride (0: one row), rows and columns."""
    if not isinstance(t, _Tensor) or t.dtype is not _INT32 or t.get_device() != index or t.dim() != 2:
        raise ValueError(f"{what} must be an int32 tensor of 2 dimensions on the tensors' device")
    (rows, width), (stride, one) = t.shape, t.stride()
    if rows < 1 or width < 1 or (width > 1 and one != 1):
        raise ValueError(f"{what} must be [rows, pages per row] with a contiguous last axis")
    return t.data_ptr(), stride if rows > 1 else 0, rows, width


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


def _out(t, like, shape, what, device):
    """The output `t`, or a new tensor like `like` (which keeps [B, N, H, d] storage), and its strides."""
    if t is None:
        t = torch.empty_like(like)
        s = t.stride()
        return t, (s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0)
    n, s = _rows(t, what, device, like.dtype)
    if n != shape:
        raise ValueError(f"{what} has another shape than its input")
    return t, s


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


def _rotary(name, q, rotary, k, positions, offset, out, k_out):
    n, qs = _rows(q, "q")
    dev, dt = q.device, q.dtype
    B, Hq, N, d = n
    if not isinstance(rotary, Rotary) or rotary.turns.device != dev:
        raise ValueError("rotary must be a Rotary on the tensors' device")
    if k is not None:
        nk, ks = _rows(k, "k", dev, dt)
        if nk[0] != B or nk[2] != N or nk[3] != d:
            raise ValueError("k must be [B, heads, N, d] with q's B, N and d")
    elif k_out is not None:
        raise ValueError("k_out without k")
    pp, pb, pn = None, 0, 0
    if positions is not None:
        if offset:
            raise ValueError("give positions or an offset, not both")
        if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32 or positions.device != dev:
            raise ValueError("positions must be an int32 tensor on the tensors' device")
        np_ = positions.shape
        if len(np_) not in (1, 2) or np_[-1] != N or (len(np_) == 2 and np_[0] != B):
            raise ValueError("positions must be int32 [N] or [B, N]")
        sp = positions.stride()
        pp, pb, pn = positions.data_ptr(), sp[0] if len(np_) == 2 else 0, sp[-1]
    if not -2 ** 31 <= offset < 2 ** 31:
        raise ValueError("offset must fit in 32 bits")
    y, ys = _out(out, q, n, "out", dev)
    z, kp, zp, Hk = None, None, None, 0
    zs = none = (0, 0, 0)
    if k is not None:
        z, zs = _out(k_out, k, nk, "k_out", dev)
        kp, zp, Hk = k.data_ptr(), z.data_ptr(), nk[1]
    opt = RotaryOptions(rotary.rotary_dim, rotary.interleaved, _DTYPES[dt], rotary.factor, rotary.turns.data_ptr(), pp, pb, pn,
                        offset, *qs, *ys, *(none if k is None else ks), *zs)
    _done(getattr(lib(), name)(q.data_ptr(), y.data_ptr(), kp, zp, B, Hq, Hk, N, d, opt, _raw_stream(dev.index)), name)
    return y if k is None else (y, z)


def _device_of(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.device


def rotary_forward(q, rotary: Rotary, k=None, positions=None, offset: int = 0, out=None, k_out=None, stream=None):
    """q [B, H, N, d] with the first rotary.rotary_dim channels of each row turned to
    its position (fa_rotary_fwd); with k [B, Hk, N, d], (q, k) in one launch.
    positions: int32 [N] or [B, N] on the device, or None for offset + n.
    out=q (k_out=k) rotates in place, also within slices of one packed projection."""
    return _on(_rotary, _device_of(q, "q"), stream, "fa_rotary_fwd", q, rotary, k, positions, int(offset), out, k_out)


def rotary_backward(dq, rotary: Rotary, dk=None, positions=None, offset: int = 0, out=None, k_out=None, stream=None):
    """Gradients with respect to rotary_forward's inputs from those of its outputs
    (fa_rotary_bwd), with the same rotary and positions: dq, or (dq, dk)."""
    return _on(_rotary, _device_of(dq, "dq"), stream, "fa_rotary_bwd", dq, rotary, dk, positions, int(offset), out, k_out)


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
        self.device, self.heads, self.page_size, self.head_dim = k.device, H, page, d
        self._struct = CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), P, H, page, d,
                                   _FORMATS[k.dtype])
        self._bytes = bytes(self._struct)  # several layers' structs are put together from these
        self._index = k.device.index

    @classmethod
    def empty(cls, num_pages: int, heads: int, head_dim: int, page_size: int = 64, dtype=torch.float8_e4m3fn, device="cuda"):
        """A pool of zeros."""
        codes = [torch.zeros((num_pages, heads, page_size, head_dim), dtype=torch.int8, device=device).view(dtype) for _ in "kv"]
        return cls(*codes, *(torch.zeros((num_pages, heads), dtype=torch.float32, device=device) for _ in "kv"))

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])


def _check_cache(cache):
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    return cache.device


def _cache_rows(name, cache, k, v, page_table, start, count):
    dev = cache.device
    n, ks = _rows(k, "k", dev)
    nv, vs = _rows(v, "v", dev, k.dtype)
    B, H, N, d = n
    if nv != n or H != cache.heads or d != cache.head_dim:
        raise ValueError("k and v must be [B, H, N, d] with the cache's H and d")
    if ks != vs:
        raise ValueError("k and v must share strides")
    rng = CacheRange(*_check_table(page_table, dev, B), _check_lengths(start, "start", dev, B),
                     _check_lengths(count, "count", dev, B), _DTYPES[k.dtype], *ks)
    _done(getattr(lib(), name)(cache._struct, k.data_ptr(), v.data_ptr(), B, N, rng, _raw_stream(dev.index)), name)


def cache_write(cache: KVCache, k, v, page_table, start, count=None, stream=None) -> None:
    """Quantises rows n < count[b] of k, v [B, H, N, d] into the cache at tokens
    start[b] + n (fa_cache_write). start, count: int32 [B]; start=None means 0,
    count=None all N rows. Where a page is shared by the old and the new tokens of a
    sequence, its older rows move to the page's new scale if that grew. The entries of
    page_table that a call writes through must name different pages. k and v share strides: where
    they are slices of one projection, rotate k in place (rotary_forward's k_out=k)."""
    _on(_cache_rows, _check_cache(cache), stream, "fa_cache_write", cache, k, v, page_table, start, count)


def cache_read(cache: KVCache, page_table, count, N: int, start=None, dtype=torch.bfloat16, k_out=None, v_out=None,
               stream=None):
    """k, v [B, H, N, d] of tokens start[b] + n, n < count[b], of the cache, in dtype
    (fa_cache_read); rows n >= count[b] are zeros."""
    return _on(_cache_read, _check_cache(cache), stream, cache, page_table, count, int(N), start, dtype, k_out, v_out)


def _cache_read(cache, page_table, count, N, start, dtype, k_out, v_out):
    dev = cache.device
    _check_int(page_table, "page_table", dev, 2)
    if N < 1:
        raise ValueError("N must be at least 1")
    if (k_out is None) != (v_out is None):
        raise ValueError("give both k_out and v_out, or neither")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be bf16 or fp16")
    shape = (page_table.shape[0], cache.heads, N, cache.head_dim)
    if k_out is None:
        k_out, v_out = torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev)
    elif k_out.dtype != dtype or tuple(k_out.shape) != shape:
        raise ValueError("k_out and v_out must be [B, H, N, d] of the call's dtype")
    _cache_rows("fa_cache_read", cache, k_out, v_out, page_table, start, count)
    return k_out, v_out


def cache_attention_workspace_bytes(cache: KVCache, B: int, heads: int, N: int, pages: int) -> int:
    """Workspace bytes with which cache_attention spreads sequences over every SM, for q
    [B, heads, N, d] and a page table of `pages` columns (0: none needed)."""
    return _on(lib().fa_cache_attention_workspace_bytes, _check_cache(cache), None, cache._struct, B, heads, N, pages)


def cache_attention(q, cache: KVCache, page_table, kv_len, q_len=None, causal: bool = True, scale: float | None = None,
                    out=None, lse=None, workspace=None, stream=None, split: bool = True):
    """O, LSE of q [B, H, N, d] over the cache's tokens j < kv_len[b] (fa_cache_attention);
    H is a multiple of the cache's heads. Causal: row i < q_len[b] (default N) sits at
    token kv_len[b] - q_len[b] + i, so the newest tokens are written before the call. Rows
    that see no token, and rows i >= q_len[b], get O = 0 and LSE = -inf. `workspace`:
    uint8 of cache_attention_workspace_bytes(...) bytes, kept by the caller, allocated
    here if None; split=False does without either."""
    return _on(_cache_attention, _check_cache(cache), stream, q, cache, page_table, kv_len, q_len, causal, scale, out, lse,
               workspace, split)


def _cache_attention(q, cache, page_table, kv_len, q_len, causal, scale, out, lse, workspace, split):
    dev = cache.device
    n, qs = _rows(q, "q", dev)
    B, H, N, d = n
    if d != cache.head_dim or H % cache.heads:
        raise ValueError("q must have the cache's d and a multiple of its heads")
    if kv_len is None:
        raise ValueError("kv_len is needed")
    table, table_stride, pages = _check_table(page_table, dev, B)
    kl, ql = _check_lengths(kv_len, "kv_len", dev, B), _check_lengths(q_len, "q_len", dev, B)
    o, os = _out(out, q, n, "out", dev)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=dev)
    elif lse.dtype != torch.float32 or lse.device != dev or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B, H, N] on the tensors' device")
    L = lib()
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the tensors' device")
        need = workspace.numel() * workspace.element_size() if split else 0
    else:
        need = L.fa_cache_attention_workspace_bytes(cache._struct, B, H, N, pages) if split else 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    opt = CacheAttentionOptions(table, table_stride, pages, kl, ql, 1 if causal else 0, _DTYPES[q.dtype],
                                d ** -0.5 if scale is None else scale, *qs, *os)
    _done(L.fa_cache_attention(q.data_ptr(), o.data_ptr(), lse.data_ptr(), cache._struct, B, H, N, opt,
                               workspace.data_ptr() if need else None, need, _raw_stream(dev.index)), "fa_cache_attention")
    return o, lse


def cache_attention_shared_workspace_bytes(cache: KVCache, B: int, heads: int, N: int, pages: int, groups: int) -> int:
    """Workspace bytes of cache_attention_shared, for q [B, heads, N, d], a page table of `pages`
    columns and `groups` groups."""
    return _on(lib().fa_cache_attention_shared_workspace_bytes, _check_cache(cache), None, cache._struct, B, heads, N, pages, groups)


def cache_attention_shared(q, cache: KVCache, page_table, kv_len, prefix_of, prefix_len, q_len=None, causal: bool = True,
                           scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """cache_attention of a batch whose sequences share prefixes, whose keys are read once for all of a
    group (fa_cache_attention_shared): the same O, LSE. prefix_of: int32 [B], each sequence's group (-1: none);
    prefix_len: int32 [groups], tokens that a group shares, in the same pages (whole pages count).
    page_table's rows and kv_len are the whole sequences', prefix included, as cache_fork
    leaves them. `workspace`: uint8 of cache_attention_shared_workspace_bytes(...) bytes, allocated here if None."""
    return _on(_cache_attention_shared, _check_cache(cache), stream, q, cache, page_table, kv_len, prefix_of, prefix_len, q_len, causal,
               scale, out, lse, workspace)


def _cache_attention_shared(q, cache, page_table, kv_len, prefix_of, prefix_len, q_len, causal, scale, out, lse, workspace):
    dev, index = cache.device, cache._index
    n, qs = _rows(q, "q", dev)
    B, H, N, d = n
    if d != cache.head_dim or H % cache.heads:
        raise ValueError("q must have the cache's d and a multiple of its heads")
    table, table_stride, rows, pages = _matrix(page_table, "page_table", index)
    if rows != B:
        raise ValueError("page_table must be [B, pages per sequence]")
    kl, of = _ints(kv_len, "kv_len", index, B), _ints(prefix_of, "prefix_of", index, B)
    ql = None if q_len is None else _ints(q_len, "q_len", index, B)
    pl, groups = _ints(prefix_len, "prefix_len", index, None), prefix_len.numel()
    o, os = _out(out, q, n, "out", dev)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=_FLOAT32, device=dev)
    elif not isinstance(lse, _Tensor) or lse.dtype is not _FLOAT32 or lse.get_device() != index or lse.shape != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B, H, N] on the tensors' device")
    L = lib()
    if workspace is None:
        need = L.fa_cache_attention_shared_workspace_bytes(cache._struct, B, H, N, pages, groups)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the tensors' device")
    else:
        need = workspace.numel() * workspace.element_size()
    opt = _OPTIONS.pack(table, table_stride, pages, kl, ql or 0, 1 if causal else 0, _DTYPES[q.dtype],
                        d ** -0.5 if scale is None else scale, *qs, *os)
    _done(L.fa_cache_attention_shared(q.data_ptr(), o.data_ptr(), lse.data_ptr(), cache._bytes, B, H, N, opt, of, pl, groups,
                                      workspace.data_ptr() if need else None, need, _raw_stream(index)), "fa_cache_attention_shared")
    return o, lse
