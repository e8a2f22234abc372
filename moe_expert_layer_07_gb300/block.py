"""Binding of what stands around the layer: the few-token layer, MXFP4 and the
norms before and after a block (declared in include/moe_gb300.h).

Argument marshalling only, as in the package's __init__: shapes and types are
read off the tensors and checked against each other here, everything else by
the library.  Where a call also takes addresses, as the package's calls do, an
integer is passed on unchecked.
"""
from __future__ import annotations

import ctypes

import torch

from . import (BF16, LAYOUT_ROWS, LAYOUT_TILES, MXFP4, OUT_BF16, OUT_F32, Config, Weights,
               _check, _CP, _I, _P, _ptr, _stream, get_device_status, lib, make_config,
               pack_expert_weights)

NORM_RMS, NORM_LAYER = 0, 1
GATE_NONE, GATE_FEATURE, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


class FewLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("status", "sched", "score", "select", "topk_ids", "topk_w", "x", "x_scales", "h",
                 "h_scales", "y", "total")]


class Norm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("hidden", "kind", "y_dtype", "residual_dtype", "param_dtype", "gate_mode")] + \
               [(n, ctypes.c_float) for n in ("eps", "residual_scale", "branch_scale")]


_SIGS = {
    "moe_layer_few_max_tokens": [],
    "moe_layer_few_workspace_size": [_CP, ctypes.POINTER(ctypes.c_size_t)],
    "moe_layer_few_layout": [_CP, ctypes.POINTER(FewLayout)],
    "moe_layer_few": [_CP, ctypes.POINTER(Weights), _I, _P, _P, _I, _P, ctypes.c_size_t, _P],
    "moe_mx4_quantize": [_I, _I, _P, _I, _P, _P, _P],
    "moe_mx4_dequantize": [_I, _I, _P, _P, _P, _I, _P],
    "moe_mx4_pack_weights": [_I, _I, _I, _P, _P, _P, _P, _P],
    "moe_mx4_grouped_gemm": [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P, _P],
    "moe_mx4_grouped_gemm_swiglu": [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P],
    "moe_block_norm": [ctypes.POINTER(Norm), _I] + [_P] * 10,
}


_OUT = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}


def _out_type(t) -> int:
    """MOE_OUT_* of a tensor."""
    kind = _OUT.get(t.dtype)
    if kind is None:
        raise TypeError(f"expected a float32 or bfloat16 tensor, got {t.dtype}")
    return kind


def _dense(t, shape, name):
    """t itself, once it is a contiguous device tensor of this shape."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor")
    return t


def _bytes(t, shape, name):
    if t.dtype is not torch.uint8:
        raise TypeError(f"{name}: expected a uint8 tensor, got {t.dtype}")
    return _dense(t, shape, name)


def _holds(t, dtype, rows, cols) -> bool:
    """Whether t has `rows` rows of `cols` elements at least (cols None: `rows` elements in any
    shape); None and addresses are the library's matter."""
    if t is None or isinstance(t, int):
        return True
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        return False
    if cols is None:
        return t.numel() >= rows
    return t.dim() > 0 and t.shape[-1] == cols and t.numel() >= rows * cols


def _check_rows(*wanted):
    """Raises for the first of (name, tensor, type, rows, columns) that does not hold."""
    for name, t, dtype, rows, cols in wanted:
        if not _holds(t, dtype, rows, cols):
            if t.dtype is not dtype:
                raise TypeError(f"{name}: expected a {dtype} tensor, got {t.dtype}")
            size = f"{rows} elements" if cols is None else f"{rows} rows of {cols}"
            raise ValueError(f"{name}: expected a contiguous CUDA tensor of {size} at least, "
                             f"got {tuple(t.shape)} on {t.device}")


# ---- MXFP4 ------------------------------------------------------------------------------


def _mx4_tensors(values, codes, scales):
    """Checks the three tensors of a quantisation; (rows, cols, type of values)."""
    shape = values.shape
    cols = shape[-1]
    kind = _OUT.get(values.dtype)
    if kind is None:
        _out_type(values)
    # one test of all that holds in a correct call; what failed is looked up after
    if not (values.is_cuda and codes.is_cuda and scales.is_cuda and values.is_contiguous()
            and codes.is_contiguous() and scales.is_contiguous() and codes.dtype is torch.uint8
            and scales.dtype is torch.uint8 and codes.shape[-1] * 2 == cols
            and scales.shape[-1] == cols // 32 and codes.shape[:-1] == shape[:-1]
            and scales.shape[:-1] == shape[:-1]):
        _dense(values, shape, "values")
        _bytes(codes, shape[:-1] + (cols // 2,), "codes")
        _bytes(scales, shape[:-1] + (cols // 32,), "scales")
    return (values.numel() // cols if cols else 0), cols, kind


def mx4_quantize(x, codes=None, scales=None, stream=None):
    """x fp32 or bf16 [..., cols] -> (codes uint8 [..., cols/2], scales uint8 [..., cols/32])."""
    if codes is None:
        codes = torch.empty(x.shape[:-1] + (x.shape[-1] // 2,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(x.shape[:-1] + (x.shape[-1] // 32,), dtype=torch.uint8, device=x.device)
    rows, cols, kind = _mx4_tensors(x, codes, scales)
    rc = lib().moe_mx4_quantize(rows, cols, x.data_ptr(), kind, codes.data_ptr(), scales.data_ptr(),
                                _stream(stream))
    if rc:
        _check(rc, "moe_mx4_quantize")
    return codes, scales


def mx4_dequantize(codes, scales, out=None, stream=None):
    """The values [..., cols] (a new bf16 tensor unless `out`, fp32 or bf16, is given)."""
    if out is None:
        out = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.bfloat16,
                          device=codes.device)
    rows, cols, kind = _mx4_tensors(out, codes, scales)
    rc = lib().moe_mx4_dequantize(rows, cols, codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
                                  kind, _stream(stream))
    if rc:
        _check(rc, "moe_mx4_dequantize")
    return out


def pack_mx4_weights(codes, scales, stream=None):
    """Row-major MXFP4 weights (codes [G, N, K/2], scales [G, N, K/32]) -> new tensors of the
    same shapes in the tile layout that the products and the few-token layer read."""
    G, N, half = codes.shape
    K = 2 * half
    _bytes(codes, (G, N, half), "codes")
    _bytes(scales, (G, N, K // 32), "scales")
    w, ws = torch.empty_like(codes), torch.empty_like(scales)
    _check(lib().moe_mx4_pack_weights(G, N, K, _ptr(codes), _ptr(scales), _ptr(w), _ptr(ws),
                                      _stream(stream)), "moe_mx4_pack_weights")
    return w, ws


_C_TYPES = {kind: dtype for dtype, kind in _OUT.items()}


def _product_fits(groups, n_out, k_dim, rows, a, a_scales, offsets, w, w_scales, status) -> bool:
    """All that holds of a correct product's operands in one test; False also for what
    _check_product would let pass (addresses, weights in other shapes of the same size)."""
    u8, i32 = torch.uint8, torch.int32
    try:
        return (a.dtype is u8 and a_scales.dtype is u8 and w.dtype is u8 and w_scales.dtype is u8
                and offsets.dtype is i32 and a.is_cuda and a_scales.is_cuda and w.is_cuda
                and w_scales.is_cuda and offsets.is_cuda and a.is_contiguous()
                and a_scales.is_contiguous() and w.is_contiguous() and w_scales.is_contiguous()
                and offsets.is_contiguous() and w.shape == (groups, n_out, k_dim // 2)
                and w_scales.shape == (groups, n_out, k_dim // 32) and a.shape[-1] == k_dim // 2
                and a_scales.shape[-1] == k_dim // 32 and a.nbytes >= rows * (k_dim // 2)
                and a_scales.nbytes >= rows * (k_dim // 32) and offsets.nbytes > 4 * groups
                and (status is None or status.dtype is i32 and status.is_cuda
                     and status.is_contiguous() and status.nbytes >= 4))
    except (AttributeError, IndexError):
        return False


def _check_product(groups, n_out, k_dim, rows, a, a_scales, offsets, w, w_scales, status, *outs):
    """Checks a grouped product's tensors against its sizes."""
    if rows <= 0:
        return
    u8, i32 = torch.uint8, torch.int32
    _check_rows(("a", a, u8, rows, k_dim // 2), ("a_scales", a_scales, u8, rows, k_dim // 32),
                ("w", w, u8, groups * n_out, k_dim // 2),
                ("w_scales", w_scales, u8, groups * n_out, k_dim // 32),
                ("expert_offsets", offsets, i32, groups + 1, None), ("status", status, i32, 1, None),
                *outs)
    for name, t in (("w", w), ("w_scales", w_scales)):
        if isinstance(t, torch.Tensor) and t.shape[-2:-1] != (n_out,):
            raise ValueError(f"{name}: expected {n_out} rows a group, got {tuple(t.shape)}")


def mx4_grouped_gemm(groups, n_out, k_dim, rows, a, a_scales, expert_offsets, w, w_scales, c,
                     c_dtype, status=None, stream=None):
    """C[r] = A[r] W[g]^T for the rows of each group; w, w_scales from pack_mx4_weights.
    a, a_scales and c may have more than `rows` rows; c is of c_dtype."""
    c_type = _C_TYPES.get(c_dtype) or getattr(c, "dtype", None)   # the library refuses other kinds
    if not (_product_fits(groups, n_out, k_dim, rows, a, a_scales, expert_offsets, w, w_scales, status)
            and _holds(c, c_type, rows, n_out)):
        _check_product(groups, n_out, k_dim, rows, a, a_scales, expert_offsets, w, w_scales,
                       status, ("c", c, c_type, rows, n_out))
    _check(lib().moe_mx4_grouped_gemm(groups, n_out, k_dim, rows, _ptr(a), _ptr(a_scales),
                                      _ptr(expert_offsets), _ptr(w), _ptr(w_scales), _ptr(c),
                                      c_dtype, _ptr(status), _stream(stream)),
           "moe_mx4_grouped_gemm")


def mx4_grouped_gemm_swiglu(groups, inter, k_dim, rows, a, a_scales, expert_offsets, w13,
                            w13_scales, h, h_scales, status=None, stream=None):
    """The gate/up product with SwiGLU, h in MXFP4 (codes [rows, inter/2], scales [rows, inter/32])."""
    u8 = torch.uint8
    if not (_product_fits(groups, 2 * inter, k_dim, rows, a, a_scales, expert_offsets, w13, w13_scales,
                          status)
            and _holds(h, u8, rows, inter // 2) and _holds(h_scales, u8, rows, inter // 32)):
        _check_product(groups, 2 * inter, k_dim, rows, a, a_scales, expert_offsets, w13, w13_scales,
                       status, ("h", h, u8, rows, inter // 2), ("h_scales", h_scales, u8, rows, inter // 32))
    _check(lib().moe_mx4_grouped_gemm_swiglu(groups, inter, k_dim, rows, _ptr(a), _ptr(a_scales),
                                             _ptr(expert_offsets), _ptr(w13), _ptr(w13_scales),
                                             _ptr(h), _ptr(h_scales), _ptr(status),
                                             _stream(stream)), "moe_mx4_grouped_gemm_swiglu")


# ---- the layer for a few tokens ------------------------------------------------------------


def layer_few_max_tokens() -> int:
    return int(lib().moe_layer_few_max_tokens())


def layer_few_workspace_size(cfg: Config) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_layer_few_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_layer_few_workspace_size")
    return n.value


def layer_few_layout(cfg: Config) -> FewLayout:
    L = FewLayout()
    _check(lib().moe_layer_few_layout(ctypes.byref(cfg), ctypes.byref(L)), "moe_layer_few_layout")
    return L


def layer_few(cfg: Config, weights: Weights, T, x, out, out_dtype, ws, ws_bytes, stream=None):
    _check(lib().moe_layer_few(ctypes.byref(cfg), ctypes.byref(weights), T, _ptr(x), _ptr(out),
                               out_dtype, _ptr(ws), ws_bytes, _stream(stream)), "moe_layer_few")


def _layer_io(x, out, out_dtype, T, hidden):
    """MOE_OUT_* of out, once x is bf16 [T, hidden] and out as large."""
    if isinstance(x, int) or isinstance(out, int):   # addresses
        return OUT_F32 if out_dtype is None else out_dtype
    kind = _OUT.get(out.dtype)
    # one test of all that holds in a correct call; what failed is looked up after
    if not (kind is not None and x.dtype is torch.bfloat16 and x.is_cuda and out.is_cuda
            and x.is_contiguous() and out.is_contiguous() and x.dim() == out.dim() == 2
            and x.shape[1] == out.shape[1] == hidden and x.shape[0] >= T and out.shape[0] >= T):
        kind = _out_type(out)
        if x.dim() != 2 or out.dim() != 2:
            raise ValueError(f"x and out: expected [{T}, {hidden}], got {tuple(x.shape)} and {tuple(out.shape)}")
        _check_rows(("x", x, torch.bfloat16, T, hidden), ("out", out, out.dtype, T, hidden))
    if out_dtype is None or out_dtype == kind:
        return kind
    if out_dtype in _C_TYPES:
        raise TypeError(f"out is {out.dtype}, and out_dtype asks for {_C_TYPES[out_dtype]}")
    return out_dtype   # refused by the library


class FewTokenLayer:
    """The MoE layer for 1 to 16 tokens a call, in two kernels.

    weights as MoELayer's; for a shape whose dtype is "mxfp4", w13 / w13_s and
    w2 / w2_s are MXFP4 codes and scale bytes as mx4_quantize gives them.
    Row-major expert weights are packed into tiles once.  An MoELayer of the
    same sizes and type may be passed in their place: its (packed) weights and
    its log2phys are then shared, also after it gets new ones (rebalancing).
    """

    def __init__(self, shape, weights, max_tokens: int | None = None, log2phys=None):
        n = layer_few_max_tokens() if max_tokens is None else max_tokens
        self.shape = shape
        self.cfg = make_config(shape, n)
        if shape.dtype == "mxfp4":
            self.cfg.dtype = MXFP4
        self._layer = weights if not isinstance(weights, dict) else None
        if self._layer is not None:
            if self._layer.expert_layout != LAYOUT_TILES:
                raise ValueError("the layer's expert weights are not packed into tiles")
            if log2phys is not None:
                raise ValueError("log2phys is the layer's own")
            for name in ("hidden", "inter", "num_experts", "num_shared", "dtype"):
                if getattr(self.cfg, name) != getattr(self._layer.cfg, name):
                    raise ValueError(f"the shape's {name} is not the layer's")
            device = self._layer.ws.device
        else:
            keep = {k: weights.get(k) for k in ("wg", "e_bias", "logit_offset", "w13", "w13_s",
                                                "w2", "w2_s", "expert_layout")}
            self._check_weights(keep)
            if keep["expert_layout"] in (None, LAYOUT_ROWS):
                for key in ("w13", "w2"):
                    if self.cfg.dtype == MXFP4:
                        keep[key], keep[key + "_s"] = pack_mx4_weights(keep[key], keep[key + "_s"])
                    else:
                        keep[key] = pack_expert_weights(self.cfg, keep[key])
            device = keep["w13"].device
            keep["log2phys"] = None if log2phys is None else torch.as_tensor(
                log2phys, dtype=torch.int32, device=device).contiguous()
            if log2phys is not None and keep["log2phys"].numel() != self.cfg.num_experts:
                raise ValueError("log2phys: expected one entry for each expert")
            self._keep = keep
            self._weights = Weights(
                w_gate=_ptr(keep["wg"]), e_bias=_ptr(keep["e_bias"]),
                logit_offset=_ptr(keep["logit_offset"]), log2phys=_ptr(keep["log2phys"]),
                w13=_ptr(keep["w13"]), w13_scales=_ptr(keep["w13_s"]), w2=_ptr(keep["w2"]),
                w2_scales=_ptr(keep["w2_s"]), expert_layout=LAYOUT_TILES)
        self.layout = layer_few_layout(self.cfg)
        self.ws_bytes = self.layout.total
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.ws[:4].zero_()   # status() before the first call

    def _check_weights(self, weights):
        """Raises for a weight tensor that is missing, or of another size than the shape says."""
        c, G = self.cfg, self.cfg.num_experts + self.cfg.num_shared
        want = {"wg": (2, (c.num_experts, c.hidden)), "e_bias": (4, (c.num_experts,)),
                "logit_offset": (4, (c.num_experts,))}
        for key, n, k in (("w13", 2 * c.inter, c.hidden), ("w2", c.hidden, c.inter)):
            if c.dtype == MXFP4:
                want[key], want[key + "_s"] = (1, (G, n, k // 2)), (1, (G, n, k // 32))
            elif c.dtype == BF16:
                want[key] = (2, (G, n, k))
            else:
                want[key], want[key + "_s"] = (1, (G, n, k)), (4, (G, n // 128, k // 128))
        for key, (size, shape) in want.items():
            t = weights[key]
            if t is None and key in ("e_bias", "logit_offset"):
                continue
            if t is None:
                raise ValueError(f"{key} is missing")
            if t.element_size() != size:
                raise TypeError(f"{key}: expected elements of {size} bytes, got {t.dtype}")
            if t.shape != shape or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{key}: expected a contiguous CUDA tensor {shape}, got "
                                 f"{tuple(t.shape)} on {t.device}")

    @property
    def weights(self) -> Weights:
        return self._layer.weights if self._layer is not None else self._weights

    def forward(self, x, out, out_dtype=None, T=None, stream=None):
        """x bf16 [T, H] and out [T, H] (fp32 or bf16) device tensors; out_dtype (OUT_*) may be
        left to out's type."""
        T = x.shape[0] if T is None else T
        out_dtype = _layer_io(x, out, out_dtype, T, self.cfg.hidden)
        layer_few(self.cfg, self.weights, T, x, out, out_dtype, self.ws, self.ws_bytes, stream)
        return out

    def view(self, name, dtype, shape):
        """A tensor view of one part of the workspace (topk_ids, topk_w, ...)."""
        import math
        off = getattr(self.layout, name)
        nbytes = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(*shape)

    def status(self) -> int:
        return get_device_status(self.ws)


# ---- norms around a block ----------------------------------------------------------------


def block_norm(residual, y=None, residual_out=None, x_out=None, w_post=None, b_post=None,
               w_pre=None, b_pre=None, gate=None, residual_scale=1.0, branch_scale=1.0, eps=1e-6,
               kind=NORM_RMS, stream=None):
    """The norm after a block, its gate and residual scale, and the norm before the next one:

        n = norm(y) w_post + b_post           (y itself without w_post)
        residual_out = residual_scale residual + branch_scale gate n
        x_out = norm(residual_out) w_pre + b_pre

    residual, y [T, H] fp32 or bf16; residual_out of residual's type (may be it), or None; x_out
    bf16, or None; gate [H], [T] or [T, H] (for T == H a one-dimensional gate is by feature)."""
    shape = residual.shape
    T, H = shape
    out = _OUT.get
    rtype = out(residual.dtype)
    ytype = OUT_F32 if y is None else out(y.dtype)
    # one test of all that holds in a correct call; what failed is looked up after
    good = rtype is not None and ytype is not None and residual.is_cuda and residual.is_contiguous()
    if y is not None:
        good = good and y.shape == shape and y.is_cuda and y.is_contiguous()
    if residual_out is not None:
        good = (good and residual_out.shape == shape and residual_out.dtype is residual.dtype
                and residual_out.is_cuda and residual_out.is_contiguous())
    if x_out is not None:
        good = (good and x_out.shape == shape and x_out.dtype is torch.bfloat16 and x_out.is_cuda
                and x_out.is_contiguous())
    mode, pdtype, row = GATE_NONE, None, (H,)
    for t in (w_post, b_post, w_pre, b_pre):
        if t is not None:
            if pdtype is None:
                pdtype = t.dtype
            good = good and t.shape == row and t.dtype is pdtype and t.is_cuda and t.is_contiguous()
    if gate is not None:
        g = gate.shape
        mode = GATE_FEATURE if g == row else GATE_TOKEN if g == (T,) else GATE_FULL
        if pdtype is None:
            pdtype = gate.dtype
        good = (good and gate.dtype is pdtype and gate.is_cuda and gate.is_contiguous()
                and (mode != GATE_FULL or g == shape))
    ptype = OUT_BF16 if pdtype is None else out(pdtype)
    if not good or ptype is None:
        _refuse_norm(shape, residual, y, residual_out, x_out, gate, mode,
                     (("w_post", w_post), ("b_post", b_post), ("w_pre", w_pre), ("b_pre", b_pre)))
    key = (H, kind, ytype, rtype, ptype, mode, eps, residual_scale, branch_scale)
    d = _NORMS.get(key)   # descriptions are plain values: made once each
    if d is None:
        if len(_NORMS) >= 256:
            _NORMS.clear()
        d = _NORMS[key] = Norm(*key)
    rc = lib().moe_block_norm(
        d, T, None if y is None else y.data_ptr(), residual.data_ptr(),
        None if gate is None else gate.data_ptr(), None if w_post is None else w_post.data_ptr(),
        None if b_post is None else b_post.data_ptr(), None if w_pre is None else w_pre.data_ptr(),
        None if b_pre is None else b_pre.data_ptr(),
        None if residual_out is None else residual_out.data_ptr(),
        None if x_out is None else x_out.data_ptr(), _stream(stream))
    if rc:
        _check(rc, "moe_block_norm")


def _refuse_norm(shape, residual, y, residual_out, x_out, gate, mode, params):
    """Raises what is wrong with block_norm's tensors."""
    for name, t in (("residual", residual), ("y", y), ("residual_out", residual_out),
                    ("x_out", x_out)):
        if t is not None:
            _out_type(_dense(t, shape, name))
    if residual_out is not None and residual_out.dtype is not residual.dtype:
        raise TypeError("residual_out must have residual's type")
    if x_out is not None and x_out.dtype is not torch.bfloat16:
        raise TypeError("x_out must be bfloat16")
    types = set()
    for name, t in params:
        if t is not None:
            types.add(_out_type(_dense(t, shape[1:], name)))
    if gate is not None:
        types.add(_out_type(_dense(gate, shape if mode == GATE_FULL else gate.shape, "gate")))
    if len(types) > 1:
        raise TypeError("norm weights, biases and gate must share one type")
    raise ValueError("block_norm: unsuitable tensors")


_NORMS: dict = {}


# ---- a decoder's MoE block ------------------------------------------------------------------


class Mx4MoELayer:
    """The MoE layer with MXFP4 experts, for any number of tokens.

    weights as FewTokenLayer's (MXFP4 codes and scale bytes, row-major), packed
    once.  Up to layer_few_max_tokens() tokens take the few-token kernels; more
    go through routing, the dispatch of bf16 rows, their quantisation, the
    grouped products and the combine.  Both quantise x and h in the same places.
    """

    def __init__(self, shape, weights: dict, max_tokens: int, log2phys=None):
        from . import permute_workspace_size
        if shape.dtype != "mxfp4":
            raise ValueError(f"expected a shape with MXFP4 experts, got {shape.dtype}")
        if not isinstance(weights, dict):
            raise TypeError("expected a dict of weights")
        self.shape = shape
        self.few = FewTokenLayer(shape, weights, log2phys=log2phys)
        self._keep = k = self.few._keep
        self.cfg = make_config(shape, max_tokens)   # routing and dispatch: bf16 rows
        self.groups = G = shape.num_experts + shape.num_shared
        T, H, I, dev = max_tokens, shape.hidden, shape.inter, k["w13"].device
        R = T * (shape.top_k + shape.num_shared)

        def buf(*size, dtype=torch.uint8):
            return torch.empty(*size, dtype=dtype, device=dev)
        i32, f32 = torch.int32, torch.float32
        self.status_word = self.few.ws[:4].view(i32)   # one word for both paths
        self.logits = buf(T, shape.num_experts, dtype=f32)
        self.ids, self.wts = buf(T, shape.top_k, dtype=i32), buf(T, shape.top_k, dtype=f32)
        self.offsets, self.src = buf(G + 1, dtype=i32), buf(R, dtype=i32)
        self.row_of_slot = buf(T, shape.top_k, dtype=i32)
        self.perm_bytes = permute_workspace_size(self.cfg, T)
        self.perm_ws = buf(max(1, self.perm_bytes))
        self.xp = buf(R, H, dtype=torch.bfloat16)
        self.xq, self.xs = buf(R, H // 2), buf(R, H // 32)
        self.h, self.hs = buf(R, I // 2), buf(R, I // 32)
        self.y = buf(R, H, dtype=f32)

    def forward(self, x, out, out_dtype=None, stream=None):
        """x bf16 [T, H] and out [T, H] (fp32 or bf16) device tensors; out_dtype (OUT_*) may be
        left to out's type."""
        from . import combine, permute, route
        T, s, k = x.shape[0], self.shape, self._keep
        if T <= self.few.cfg.max_tokens:
            return self.few.forward(x, out, out_dtype, stream=stream)
        if T > self.cfg.max_tokens:
            raise ValueError(f"{T} tokens, and buffers for {self.cfg.max_tokens}")
        out_dtype = _layer_io(x, out, out_dtype, T, s.hidden)
        rows = T * (s.top_k + s.num_shared)
        st = self.status_word
        layer_few(self.few.cfg, self.few.weights, 0, None, None, OUT_F32, self.few.ws,
                  self.few.ws_bytes, stream)   # no tokens: zeroes the word
        route(self.cfg, T, x, k["wg"], k["e_bias"], k["logit_offset"], k["log2phys"], self.logits,
              self.ids, self.wts, st, stream)
        permute(self.cfg, T, self.ids, x, None, self.offsets, self.src, self.row_of_slot, self.xp,
                None, self.perm_ws, self.perm_bytes, st, stream)
        mx4_quantize(self.xp[:rows], self.xq[:rows], self.xs[:rows], stream)
        mx4_grouped_gemm_swiglu(self.groups, s.inter, s.hidden, rows, self.xq, self.xs, self.offsets,
                                k["w13"], k["w13_s"], self.h, self.hs, st, stream)
        mx4_grouped_gemm(self.groups, s.hidden, s.inter, rows, self.h, self.hs, self.offsets,
                         k["w2"], k["w2_s"], self.y, OUT_F32, st, stream)
        combine(self.cfg, T, self.y, self.row_of_slot, self.wts, self.offsets, out, out_dtype, stream)
        return out

    def status(self) -> int:
        """The device status of the last call, as MoELayer's."""
        return self.few.status()


class MoEBlock:
    """x = norm(r) w_pre;  y = layer(x);  r = residual_scale r + branch_scale gate norm(y) w_post.

    layer: an MoELayer, a FewTokenLayer or an Mx4MoELayer.  With `few` (a
    FewTokenLayer) calls of few tokens go there.  w_post and gate may be None.
    kind may be NORM_LAYER; norms with biases are block_norm's alone.
    """

    def __init__(self, layer, w_pre, w_post=None, gate=None, residual_scale=1.0, branch_scale=1.0,
                 eps=1e-6, kind=NORM_RMS, few: FewTokenLayer | None = None):
        self.layer, self.few = layer, few
        self.w_pre, self.w_post, self.gate = w_pre, w_post, gate
        self.scales = dict(residual_scale=residual_scale, branch_scale=branch_scale)
        self.norm = dict(eps=eps, kind=kind)

    def pre(self, residual, x, stream=None):
        """x = norm(residual) w_pre, where no earlier block wrote it."""
        block_norm(residual, x_out=x, w_pre=self.w_pre, stream=stream, **self.norm)
        return x

    def forward(self, residual, x, y, w_next=None, x_next=None, stream=None):
        """residual fp32 or bf16 [T, H], updated in place; x bf16 [T, H] the normed input (from
        `pre`, or the block before); y bf16 [T, H] is scratch.  With w_next the next block's
        norm is part of the same pass, into x_next (may be x)."""
        few = self.few is not None and x.shape[0] <= self.few.cfg.max_tokens
        (self.few if few else self.layer).forward(x, y, OUT_BF16, stream=stream)
        block_norm(residual, y=y, residual_out=residual, x_out=x_next, w_post=self.w_post,
                   w_pre=w_next, gate=self.gate, stream=stream, **self.scales, **self.norm)
        return residual
