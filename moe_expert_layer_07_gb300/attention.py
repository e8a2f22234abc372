"""Binding of attention's half of a decoder layer, over a cache in four bits (declared in
include/moe_gb300.h): the tables of its pages, the norm and rotation of queries and keys with the
cache's write, the attention, and products of a few rows with four-bit weights.

Argument marshalling only, as in block.py: shapes and types are read off the tensors and checked
against each other here, everything else by the library.
"""
from __future__ import annotations

import copy
import ctypes

import torch

from . import DEV_BAD_INDEX, OUT_BF16, OUT_F32, _check, _I, _P, _stream, lib
from .block import _OUT, NORM_RMS, _dense, block_norm, mx4_grouped_gemm, mx4_quantize, pack_mx4_weights

ROPE_HALVES, ROPE_PAIRS = 0, 1
W4_MX, W4_INT = 0, 1


class _Cache(ctypes.Structure):
    _fields_ = [("codes", _P), ("scales", _P)] + \
               [(n, ctypes.c_int32) for n in ("pages", "kv_heads", "page", "dim")]


class _Rope(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("q_heads", "kv_heads", "dim", "rope_dim", "style", "param_dtype", "max_positions",
                 "qkv_stride")] + [("eps", ctypes.c_float)]


class _Attn(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("requests", "rows", "q_heads", "max_pages", "max_q", "max_len", "window")] + \
               [("scale", ctypes.c_float)]


class _W4(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_out", "k_dim", "kind", "group", "scale_dtype")]


_CACHE = ctypes.POINTER(_Cache)
_SIGS = {
    "moe_cache_tables": [_I, _I, _P, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _I, _P, _P, _P],
    "moe_qk_norm_rope": [ctypes.POINTER(_Rope), _I] + [_P] * 7 + [_CACHE, _P, _P, _P],
    "moe_cache_read": [_CACHE, _I] + [_P] * 5,
    "moe_cache_attention_workspace_size": [ctypes.POINTER(_Attn), _CACHE, ctypes.POINTER(ctypes.c_size_t)],
    "moe_cache_attention": [ctypes.POINTER(_Attn), _CACHE, _P, _P, _P, _P, _P, _I, _P, _P, ctypes.c_size_t,
                            _P, _P],
    "moe_w4_matvec": [ctypes.POINTER(_W4), _I, _P, _P, _P, _P, _P, _I, _P],
}

_I32, _BF16 = torch.int32, torch.bfloat16


def _at(t):
    return None if t is None else t.data_ptr()


def _typed(t, dtype, shape, name):
    """t itself, once it is a contiguous device tensor of this type and shape."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected a {dtype} tensor, got {t.dtype}")
    return _dense(t, shape, name)


# torch's raw queries, as in __init__.py; the public ones cost microseconds of a small call
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_ELSEWHERE = "expected tensors of one device, the current one"


def _word(status, dev):
    if status.dtype is not _I32 or status.numel() < 1 or status.get_device() != dev:
        raise TypeError("status: expected an int32 CUDA tensor on the others' device")
    return status.data_ptr()


class Cache4:
    """Keys and values of kv_heads heads of `dim` channels in MXFP4, in pages of `page` tokens:
    codes uint8 [pages, 2, kv_heads, page, dim/2], scales uint8 [pages, 2, kv_heads, page, dim/32].
    What no token was written to may hold anything."""

    def __init__(self, pages, page, kv_heads, dim, device="cuda"):
        self._set(torch.empty(pages, 2, kv_heads, page, dim // 2, dtype=torch.uint8, device=device),
                  torch.empty(pages, 2, kv_heads, page, dim // 32, dtype=torch.uint8, device=device))

    @classmethod
    def of(cls, codes, scales):
        """A cache in tensors that are there."""
        self = cls.__new__(cls)
        self._set(codes, scales)
        return self

    def _set(self, codes, scales):
        if codes.dim() != 5 or codes.shape[1] != 2:
            raise ValueError(f"codes: expected [pages, 2, kv_heads, page, dim/2], got {tuple(codes.shape)}")
        pages, _, kv_heads, page, half = codes.shape
        if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
            raise TypeError("codes and scales: expected uint8 tensors")
        _dense(codes, codes.shape, "codes")
        _dense(scales, (pages, 2, kv_heads, page, half // 16), "scales")
        self.device = codes.get_device()
        if scales.get_device() != self.device:
            raise ValueError(_ELSEWHERE)
        self.codes, self.scales = codes, scales
        self.pages, self.page, self.kv_heads, self.dim = pages, page, kv_heads, 2 * half
        self.c = _Cache(codes.data_ptr(), scales.data_ptr(), pages, kv_heads, page, 2 * half)


def rope_table(max_positions, rope_dim, base=10000.0, device="cuda"):
    """fp32 [max_positions, rope_dim]: the cosines of the angles position * base^(-2i / rope_dim),
    then their sines, formed in 64 bits."""
    freq = float(base) ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def cache_tables(held, new_tokens, free_pages, free_range, page, table, lengths, starts, slots, positions,
                 free_out, status=None, stream=None):
    """Tables of one step: request b holds held[b] tokens and gets new_tokens[b] more.

    Its new pages are taken from the ring free_pages, whose entries free_range[0] .. free_range[1]-1
    (mod its size) are free, and written behind those that its row of `table` has.  lengths (may be
    held), starts [B+1], slots and positions [any number of token rows; -1 and 0 behind the last
    token] and free_out (may be free_range) are written.  A step for which pages, columns or rows do
    not suffice is not made: see moe_cache_tables."""
    B, w = held.shape[0], table.shape[1] if table.dim() == 2 else -1
    n, f = slots.shape[0], free_pages.shape[0]
    i64 = torch.int64
    # one test of all that holds in a correct call; what failed is looked up after
    dev = held.get_device()
    good = dev >= 0
    for t in (held, new_tokens, free_pages, table, lengths, starts, slots, positions):
        good = good and t.dtype is _I32 and t.get_device() == dev and t.is_contiguous()
    if not (good and free_range.dtype is i64 and free_out.dtype is i64 and dev == free_range.get_device()
            and dev == free_out.get_device() and dev == _current_device() and free_range.is_contiguous()
            and free_out.is_contiguous() and free_range.shape == free_out.shape == (2,)
            and held.shape == new_tokens.shape == lengths.shape == (B,) and table.shape == (B, w)
            and starts.shape == (B + 1,) and slots.shape == positions.shape == (n,)
            and free_pages.shape == (f,)):
        for name, t, shape in (("held", held, (B,)), ("new_tokens", new_tokens, (B,)),
                               ("free_pages", free_pages, (f,)), ("table", table, (B, w)),
                               ("lengths", lengths, (B,)), ("starts", starts, (B + 1,)),
                               ("slots", slots, (n,)), ("positions", positions, (n,))):
            _typed(t, _I32, shape, name)
        _typed(free_range, i64, (2,), "free_range")
        _typed(free_out, i64, (2,), "free_out")
        raise ValueError(_ELSEWHERE)
    word = None if status is None else _word(status, dev)
    s = _raw_stream(dev) if stream is None else _stream(stream)
    rc = lib().moe_cache_tables(B, page, held.data_ptr(), new_tokens.data_ptr(), free_pages.data_ptr(), f,
                                free_range.data_ptr(), table.data_ptr(), w, lengths.data_ptr(),
                                starts.data_ptr(), slots.data_ptr(), positions.data_ptr(), n,
                                free_out.data_ptr(), word, s)
    if rc:
        _check(rc, "moe_cache_tables")


def qk_norm_rope(qkv, positions, cos_sin, q_heads, kv_heads, q_out, k_out=None, w_q=None, w_k=None,
                 cache: Cache4 | None = None, slots=None, eps=1e-6, style=ROPE_HALVES, status=None,
                 stream=None):
    """Norm (with w_q, w_k) and rotation of each head's queries and keys; keys to k_out, or with the
    values to `slots` of the cache, or both.

    qkv bf16 [T, at least (q_heads + 2 kv_heads) dim], rows a multiple of 8 elements apart, positions int32 [T], cos_sin
    fp32 [positions, rope_dim] as rope_table gives it (None: no rotation), q_out bf16 [T, q_heads, dim],
    k_out bf16 [T, kv_heads, dim], w_* [dim] fp32 or bf16, slots int32 [T] (-1: nowhere)."""
    T, dim = qkv.shape[0], q_out.shape[-1]
    width = (q_heads + 2 * kv_heads) * dim
    rot = 0 if cos_sin is None else cos_sin.shape[-1]
    param = w_q if w_q is not None else w_k
    pkind = OUT_BF16 if param is None else _OUT.get(param.dtype)
    # one test of all that holds in a correct call; what failed is looked up after
    dev = qkv.get_device()
    good = (pkind is not None and qkv.dtype is _BF16 and q_out.dtype is _BF16 and dev >= 0
            and q_out.get_device() == dev and dev == _current_device() and qkv.dim() == 2 and qkv.stride(1) == 1
            and qkv.shape[1] >= width and (T < 2 or qkv.stride(0) < 2 ** 31)
            and q_out.shape == (T, q_heads, dim) and q_out.is_contiguous() and (cache is None) == (slots is None))
    for w in (w_q, w_k):
        if w is not None:
            good = (good and w.dtype is param.dtype and w.shape == (dim,) and w.get_device() == dev
                    and w.is_contiguous())
    if k_out is not None:
        good = (good and k_out.dtype is _BF16 and k_out.shape == (T, kv_heads, dim)
                and k_out.get_device() == dev and k_out.is_contiguous())
    if rot:
        good = (good and cos_sin.dtype is torch.float32 and cos_sin.dim() == 2 and cos_sin.get_device() == dev
                and cos_sin.is_contiguous() and positions.dtype is _I32 and positions.shape == (T,)
                and positions.get_device() == dev and positions.is_contiguous())
    if slots is not None:
        good = (good and slots.dtype is _I32 and slots.shape == (T,) and slots.get_device() == dev
                and slots.is_contiguous() and cache.device == dev)
    if not good:
        _refuse_rope(qkv, positions, cos_sin, rot, q_heads, kv_heads, q_out, k_out, w_q, w_k, param, pkind, cache, slots)
    stride = qkv.stride(0) if T > 1 else width   # (of one row it says nothing)
    key = (q_heads, kv_heads, dim, rot, style, pkind, cos_sin.shape[0] if rot else 0, stride, eps)
    d = _ROPES.get(key)   # descriptions are plain values: made once each
    if d is None:
        if len(_ROPES) >= 256:
            _ROPES.clear()
        d = _ROPES[key] = _Rope(*key)
    word = None if status is None else _word(status, dev)
    s = _raw_stream(dev) if stream is None else _stream(stream)
    rc = lib().moe_qk_norm_rope(d, T, qkv.data_ptr(), _at(positions), _at(cos_sin) if rot else None, _at(w_q),
                                _at(w_k), q_out.data_ptr(), _at(k_out), None if cache is None else cache.c,
                                _at(slots), word, s)
    if rc:
        _check(rc, "moe_qk_norm_rope")


def _refuse_rope(qkv, positions, cos_sin, rot, q_heads, kv_heads, q_out, k_out, w_q, w_k, param, pkind, cache, slots):
    """Raises what is wrong with qk_norm_rope's tensors."""
    T, dim = qkv.shape[0], q_out.shape[-1]
    if qkv.dtype is not _BF16:
        raise TypeError(f"qkv: expected a bfloat16 tensor, got {qkv.dtype}")
    _typed(q_out, _BF16, (T, q_heads, dim), "q_out")
    if pkind is None:
        raise TypeError(f"w_q, w_k: expected float32 or bfloat16 tensors, got {param.dtype}")
    for name, w in (("w_q", w_q), ("w_k", w_k)):
        if w is not None:
            _typed(w, param.dtype, (dim,), name)
    if k_out is not None:
        _typed(k_out, _BF16, (T, kv_heads, dim), "k_out")
    if rot:
        _typed(cos_sin, torch.float32, (cos_sin.shape[0], rot), "cos_sin")
        _typed(positions, _I32, (T,), "positions")
    if (cache is None) != (slots is None):
        raise ValueError("cache and slots go together")
    if slots is not None:
        _typed(slots, _I32, (T,), "slots")
    if T > 1 and qkv.dim() == 2 and qkv.stride(0) >= 2 ** 31:
        raise ValueError(f"qkv: rows are {qkv.stride(0)} elements apart, and 2^31 - 1 at most may be")
    if qkv.is_cuda and qkv.dim() == 2 and qkv.stride(1) == 1 and qkv.shape[1] >= (q_heads + 2 * kv_heads) * dim:
        raise ValueError(_ELSEWHERE)
    raise ValueError(f"qkv: expected CUDA rows of {q_heads} + 2 x {kv_heads} heads of {dim}, got {tuple(qkv.shape)}")


_ROPES: dict = {}


def cache_read(cache: Cache4, slots, k=None, v=None, status=None, stream=None):
    """The values in `slots` of the cache: k, v bf16 [n, kv_heads, dim], either may be None.  Rows of
    slot -1 are left as they were."""
    n = slots.shape[0]
    shape = (n, cache.kv_heads, cache.dim)
    dev = cache.device
    good = (slots.dtype is _I32 and slots.shape == (n,) and slots.get_device() == dev and slots.is_contiguous()
            and dev == _current_device())
    for t in (k, v):
        if t is not None:
            good = good and t.dtype is _BF16 and t.shape == shape and t.get_device() == dev and t.is_contiguous()
    if not good:
        _typed(slots, _I32, (n,), "slots")
        for name, t in (("k", k), ("v", v)):
            if t is not None:
                _typed(t, _BF16, shape, name)
        raise ValueError(_ELSEWHERE)
    word = None if status is None else _word(status, dev)
    s = _raw_stream(dev) if stream is None else _stream(stream)
    rc = lib().moe_cache_read(cache.c, n, slots.data_ptr(), _at(k), _at(v), word, s)
    if rc:
        _check(rc, "moe_cache_read")


class CacheAttention:
    """Attention of up to `rows` query rows of up to `requests` requests over a cache, with the
    workspace that it needs (one call at a time).

    max_q: the most query tokens of one request, max_pages: columns of the page table; max_len: the longest
    request (nothing is chosen by it).  max_q chooses the kernels and is no limit: where max_q tokens have
    more than 32 rows (tokens times heads of a KV head) the kernels for many rows are launched in every call, and
    without that requests of many rows take several times as long.  window: how many tokens a query sees,
    itself included (0: all)."""

    def __init__(self, requests, rows, q_heads, cache: Cache4, max_pages, max_q=1, max_len=None, window=0,
                 scale=None):
        self.cache = cache
        self.d = _Attn(requests, rows, q_heads, max_pages, max_q,
                       max_pages * cache.page if max_len is None else max_len, window,
                       cache.dim ** -0.5 if scale is None else scale)
        n = ctypes.c_size_t()
        _check(lib().moe_cache_attention_workspace_size(self.d, cache.c, ctypes.byref(n)),
               "moe_cache_attention_workspace_size")
        self.ws_bytes = n.value
        self.ws = torch.empty(max(1, n.value), dtype=torch.uint8, device=cache.codes.device)

    def of_rows(self, rows):
        """The same for fewer query rows, in the same workspace."""
        d = self.d
        if not 0 <= rows <= d.rows:
            raise ValueError(f"{rows} rows, and a workspace for {d.rows}")
        other = copy.copy(self)
        other.d = _Attn(d.requests, rows, d.q_heads, d.max_pages, d.max_q, d.max_len, d.window, d.scale)
        return other

    def forward(self, q, table, lengths, starts, out, lse=None, status=None, stream=None):
        """q bf16 [rows, q_heads, dim], out the same in bf16 (may be q) or fp32; table int32 [requests,
        max_pages], lengths int32 [requests], starts int32 [requests + 1] as cache_tables writes them;
        lse fp32 [rows, q_heads] or None.  Rows behind the last request are left as they were."""
        d, c = self.d, self.cache
        dev = c.device
        shape = (d.rows, d.q_heads, c.dim)
        kind = _OUT.get(out.dtype)
        # one test of all that holds in a correct call; what failed is looked up after
        if not (kind is not None and q.dtype is _BF16 and q.shape == out.shape == shape and q.get_device() == dev
                and out.get_device() == dev and dev == _current_device()
                and q.is_contiguous() and out.is_contiguous() and table.dtype is _I32 and lengths.dtype is _I32
                and starts.dtype is _I32 and table.get_device() == dev and lengths.get_device() == dev
                and starts.get_device() == dev
                and table.is_contiguous() and lengths.is_contiguous() and starts.is_contiguous()
                and table.shape == (d.requests, d.max_pages) and lengths.shape == (d.requests,)
                and starts.shape == (d.requests + 1,)
                and (lse is None or lse.dtype is torch.float32 and lse.shape == shape[:2]
                     and lse.get_device() == dev and lse.is_contiguous())):
            _typed(q, _BF16, shape, "q")
            if kind is None:
                raise TypeError(f"out: expected a float32 or bfloat16 tensor, got {out.dtype}")
            _dense(out, shape, "out")
            _typed(table, _I32, (d.requests, d.max_pages), "table")
            _typed(lengths, _I32, (d.requests,), "lengths")
            _typed(starts, _I32, (d.requests + 1,), "starts")
            if lse is not None:
                _typed(lse, torch.float32, shape[:2], "lse")
            raise ValueError(_ELSEWHERE)
        word = None if status is None else _word(status, dev)
        s = _raw_stream(dev) if stream is None else _stream(stream)
        rc = lib().moe_cache_attention(d, c.c, q.data_ptr(), table.data_ptr(), lengths.data_ptr(),
                                       starts.data_ptr(), out.data_ptr(), kind, _at(lse), self.ws.data_ptr(),
                                       self.ws_bytes, word, s)
        if rc:
            _check(rc, "moe_cache_attention")
        return out


def w4_matvec(x, codes, scales, out, zeros=None, stream=None):
    """out = x W^T for 1 to 16 rows: x bf16 [T, K], out fp32 or bf16 [T, N], codes uint8 [N, K/2] (the even
    element in the low four bits).  scales uint8 [N, K/32]: W in MXFP4, as mx4_quantize gives it;
    scales fp32 or bf16 [N, K/group]: W = scales (codes - zeros), group 32, 64 or 128, zeros uint8
    [N, K/group] or None (8)."""
    T, K = x.shape
    N = codes.shape[0]
    kind, skind = _OUT.get(out.dtype), _OUT.get(scales.dtype)
    mx = scales.dtype is torch.uint8
    groups = scales.shape[-1]
    dev = x.get_device()
    if not (kind is not None and (mx or skind is not None) and x.dtype is _BF16 and codes.dtype is torch.uint8
            and dev >= 0 and codes.get_device() == dev and scales.get_device() == dev and out.get_device() == dev
            and dev == _current_device() and x.is_contiguous()
            and codes.is_contiguous() and scales.is_contiguous() and out.is_contiguous()
            and codes.shape == (N, K // 2) and out.shape == (T, N) and groups and K % groups == 0
            and scales.shape == (N, groups)
            and (zeros is None or not mx and zeros.dtype is torch.uint8 and zeros.shape == scales.shape
                 and zeros.get_device() == dev and zeros.is_contiguous())):
        _typed(x, _BF16, (T, K), "x")
        _typed(codes, torch.uint8, (N, K // 2), "codes")
        if kind is None:
            raise TypeError(f"out: expected a float32 or bfloat16 tensor, got {out.dtype}")
        _dense(out, (T, N), "out")
        if not mx and skind is None:
            raise TypeError(f"scales: expected a uint8, float32 or bfloat16 tensor, got {scales.dtype}")
        _dense(scales, (N, groups), "scales")
        if not groups or K % groups:
            raise ValueError(f"scales: {groups} groups do not divide {K}")
        if zeros is not None:
            if mx:
                raise ValueError("MXFP4 has no zero points")
            _typed(zeros, torch.uint8, (N, groups), "zeros")
        raise ValueError(_ELSEWHERE)
    key = (N, K, W4_MX if mx else W4_INT, K // groups, OUT_F32 if mx else skind)
    d = _W4S.get(key)
    if d is None:
        if len(_W4S) >= 256:
            _W4S.clear()
        d = _W4S[key] = _W4(*key)
    s = _raw_stream(dev) if stream is None else _stream(stream)
    rc = lib().moe_w4_matvec(d, T, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), _at(zeros),
                             out.data_ptr(), kind, s)
    if rc:
        _check(rc, "moe_w4_matvec")
    return out


_W4S: dict = {}


# ---- a decoder's attention block ---------------------------------------------------------------


class PageTables:
    """The tables of a cache's pages for up to `requests` requests, on the GPU: step() takes the
    requests one step on, in one launch that a CUDA graph can hold.

    lengths int32 [requests], table int32 [requests, max_pages], and of the step: starts
    [requests + 1], slots and positions [max_tokens].  status: the device status word."""

    def __init__(self, cache: Cache4, requests, max_pages, max_tokens):
        dev = cache.codes.device
        zeros = lambda *n: torch.zeros(*n, dtype=_I32, device=dev)  # noqa: E731
        self.page = cache.page
        self.lengths, self.table = zeros(requests), zeros(requests, max_pages)
        self.starts, self.slots, self.positions = zeros(requests + 1), zeros(max_tokens), zeros(max_tokens)
        self.free_pages = torch.arange(cache.pages, dtype=_I32, device=dev)
        self.free_range = torch.tensor([0, cache.pages], dtype=torch.int64, device=dev)
        self.status = zeros(1)

    def step(self, new_tokens, stream=None):
        """new_tokens int32 [requests]: how many tokens each request gets."""
        cache_tables(self.lengths, new_tokens, self.free_pages, self.free_range, self.page, self.table,
                     self.lengths, self.starts, self.slots, self.positions, self.free_range, self.status, stream)

    def release(self, request, length=None):
        """Gives the pages of a request back; it holds none then.  On the current stream, between steps, without
        waiting for it: the pages are those of lengths[request].  length: what the caller takes it to hold; a
        number that is not as many pages sets DEV_BAD_INDEX in status."""
        if not 0 <= request < self.lengths.shape[0]:
            raise IndexError(f"request {request} of {self.lengths.shape[0]}")
        ring = self.free_pages.shape[0]
        i = torch.arange(min(ring, self.table.shape[1]), device=self.free_pages.device)
        n = (self.lengths[request] + (self.page - 1)) // self.page
        if i.shape[0]:
            at = (self.free_range[1] + i) % ring
            self.free_pages[at] = torch.where(i < n, self.table[request, :i.shape[0]], self.free_pages[at])
        self.free_range[1] += n
        if length is not None:
            self.status |= (n != -(-length // self.page)).int() * DEV_BAD_INDEX
        self.lengths[request] = 0


class AttentionBlock:
    """q, k, v = x W_qkv;  q, k normed and rotated, k and v into the cache;  o = attention;
    r = residual_scale r + branch_scale gate norm(o W_o) w_post: the attention half of a decoder
    layer, beside MoEBlock.

    w_qkv, w_o: MXFP4 (codes [N, K/2], scale bytes [N, K/32], row-major, as mx4_quantize gives them) of
    [(q_heads + 2 kv_heads) dim, hidden] and [hidden, q_heads dim].  Up to 16 rows are multiplied in bf16
    (w4_matvec); more, a prompt's, are quantised to MXFP4 themselves (mx4_grouped_gemm on packed
    copies, made where max_rows is more than 16: both sizes then multiples of 128): from 17 rows on
    projections carry the error of four bits on both sides.  max_q: the most tokens that one request gets in
    any step, one choice for all of them (CacheAttention): max_rows for prompts, 1 where the block only decodes.
    One call at a time."""

    def __init__(self, cache: Cache4, q_heads, hidden, w_qkv, w_o, cos_sin, requests, max_rows, max_pages, max_q=1,
                 max_len=None, w_q=None, w_k=None, w_pre=None, w_post=None, gate=None, residual_scale=1.0,
                 branch_scale=1.0, eps=1e-6, kind=NORM_RMS, style=ROPE_HALVES, window=0, scale=None):
        self.cache, self.q_heads, self.hidden, self.cos_sin = cache, q_heads, hidden, cos_sin
        self.max_rows = max_rows
        self.plan = CacheAttention(requests, max_rows, q_heads, cache, max_pages, max_q, max_len, window, scale)
        self.w_q, self.w_k, self.w_pre, self.w_post, self.gate = w_q, w_k, w_pre, w_post, gate
        self.eps, self.kind, self.style = eps, kind, style
        self.scales = dict(residual_scale=residual_scale, branch_scale=branch_scale)
        D, n_qkv = cache.dim, (q_heads + 2 * cache.kv_heads) * cache.dim
        dev = cache.codes.device
        self.weights, self.sizes = (w_qkv, w_o), ((n_qkv, hidden), (hidden, q_heads * D))
        for name, (codes, scales), (n, k) in zip(("w_qkv", "w_o"), self.weights, self.sizes):
            _typed(codes, torch.uint8, (n, k // 2), name)
            _typed(scales, torch.uint8, (n, k // 32), name)
        self.packed = None
        if max_rows > 16:
            self.packed = [pack_mx4_weights(c[None], s[None]) for c, s in self.weights]
            k = max(hidden, q_heads * D)
            self.xq = torch.empty(max_rows * k // 2, dtype=torch.uint8, device=dev)
            self.xs = torch.empty(max_rows * k // 32, dtype=torch.uint8, device=dev)
            self.offsets = torch.zeros(max_rows + 1, 4, dtype=_I32, device=dev)   # row T: 0, T
            self.offsets[:, 1] = torch.arange(max_rows + 1, device=dev)
        self.qkv = torch.empty(max_rows, n_qkv, dtype=_BF16, device=dev)
        self.q = torch.zeros(max_rows, q_heads, D, dtype=_BF16, device=dev)
        self.status_word = torch.zeros(1, dtype=_I32, device=dev)
        self._plans = {}

    def _project(self, which, x, out, stream):
        (n, k), T = self.sizes[which], x.shape[0]
        if T <= 16:
            return w4_matvec(x, *self.weights[which], out, stream=stream)
        xq, xs = self.xq[:T * k // 2].view(T, k // 2), self.xs[:T * k // 32].view(T, k // 32)
        mx4_quantize(x, xq, xs, stream)
        mx4_grouped_gemm(1, n, k, T, xq, xs, self.offsets[T], *self.packed[which], out, OUT_BF16, self.status_word,
                         stream)
        return out

    def pre(self, residual, x, stream=None):
        """x = norm(residual) w_pre, where no earlier block wrote it."""
        block_norm(residual, x_out=x, w_pre=self.w_pre, eps=self.eps, kind=self.kind, stream=stream)
        return x

    def forward(self, residual, x, y, tables: PageTables, w_next=None, x_next=None, stream=None):
        """residual fp32 or bf16 [T, hidden], updated in place; x bf16 [T, hidden] the normed input; y
        bf16 [T, hidden] is scratch; tables: of this step, for a cache of the same page size, with at most T
        token rows (rows behind the last token go nowhere; what their outputs hold means nothing).  With w_next the next block's
        norm is part of the last pass, into x_next (may be x)."""
        T = x.shape[0]
        if T > self.max_rows:
            raise ValueError(f"{T} rows, and buffers for {self.max_rows}")
        if tables.slots.shape[0] < T:
            raise ValueError(f"{T} rows, and tables for {tables.slots.shape[0]}")
        if tables.page != self.cache.page:
            raise ValueError(f"a cache in pages of {self.cache.page}, and tables of pages of {tables.page}")
        if tables.table.shape != (self.plan.d.requests, self.plan.d.max_pages):
            raise ValueError(f"tables of {tuple(tables.table.shape)} requests and pages, and a block for "
                             f"{(self.plan.d.requests, self.plan.d.max_pages)}")
        plan = self._plans.get(T)
        if plan is None:
            plan = self._plans[T] = self.plan.of_rows(T)
        qkv, q = self.qkv[:T], self.q[:T]
        self._project(0, x, qkv, stream)
        qk_norm_rope(qkv, tables.positions[:T], self.cos_sin, self.q_heads, self.cache.kv_heads, q, w_q=self.w_q,
                     w_k=self.w_k, cache=self.cache, slots=tables.slots[:T], eps=self.eps, style=self.style,
                     status=self.status_word, stream=stream)
        plan.forward(q, tables.table, tables.lengths, tables.starts, q, status=self.status_word, stream=stream)
        self._project(1, q.view(T, -1), y, stream)
        block_norm(residual, y=y, residual_out=residual, x_out=x_next, w_post=self.w_post, w_pre=w_next,
                   gate=self.gate, eps=self.eps, kind=self.kind, stream=stream, **self.scales)
        return residual

    def status(self) -> int:
        """The device status bits of the calls so far (waits for them)."""
        return int(self.status_word)
