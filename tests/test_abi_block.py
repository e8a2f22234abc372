"""The entry points around the layer on the host (no GPU needed): every refusal comes before any
launch, sizes and layouts are what the header says."""
import ctypes
import dataclasses

import pytest

import moe_expert_layer_07_gb300 as moe
import synth

P = ctypes.c_void_p
FAKE, ODD, MIS16 = P(0x1000), P(0x1008), P(0x1010)   # never dereferenced; MIS16 is not 32-aligned


@pytest.fixture(scope="module")
def L():
    from moe_expert_layer_07_gb300 import _build
    _build.build()
    return moe.lib()


def _cfg(**kw):
    cfg = moe.make_config(synth.CONFIGS["r1_mini"], 16)
    for k, v in kw.items():
        setattr(cfg, k, v)
    return cfg


def _weights(**kw):
    d = dict(w_gate=0x1000, e_bias=None, logit_offset=None, log2phys=None, w13=0x1000,
             w13_scales=0x1000, w2=0x1000, w2_scales=0x1000, expert_layout=moe.LAYOUT_TILES)
    d.update(kw)
    return moe.Weights(**d)


def test_few_workspace(L):
    assert moe.layer_few_max_tokens() == 16
    for dtype in (moe.BF16, moe.FP8, moe.MXFP4):
        cfg = _cfg(dtype=dtype)
        lay = moe.layer_few_layout(cfg)
        assert lay.total == moe.layer_few_workspace_size(cfg) and lay.status == 0
        offs = [getattr(lay, n) for n, _ in lay._fields_]
        assert offs == sorted(offs) and all(o % 256 == 0 for o in offs)
        rows = 16 * 9
        assert lay.total - lay.y == rows * cfg.hidden * 4
    # h: two bf16 parts, segments of 128 values and a scale, packed codes
    size = {d: moe.layer_few_layout(_cfg(dtype=d)) for d in (moe.BF16, moe.FP8, moe.MXFP4)}
    assert size[moe.BF16].h_scales - size[moe.BF16].h == 16 * 9 * 384 * 4
    assert size[moe.MXFP4].h_scales - size[moe.MXFP4].h == 16 * 9 * 384 // 2


def test_few_refusals(L):
    n = ctypes.c_size_t()
    need = moe.layer_few_workspace_size(_cfg())

    def call(cfg=None, w=None, T=4, x=FAKE, out=FAKE, kind=0, ws=FAKE, size=need):
        return L.moe_layer_few(ctypes.byref(cfg or _cfg()), ctypes.byref(w or _weights()), T, x, out,
                               kind, ws, size, None)
    assert L.moe_layer_few_workspace_size(None, ctypes.byref(n)) == -1
    assert L.moe_layer_few_workspace_size(ctypes.byref(_cfg()), None) == -1
    assert call(cfg=_cfg(max_tokens=17)) == -2
    assert call(cfg=_cfg(dtype=3)) == -1
    assert call(cfg=_cfg(hidden=1000)) == -2
    assert call(cfg=_cfg(top_k=17)) == -2
    assert call(T=17) == -1 and call(T=-1) == -1
    assert call(x=None) == -1 and call(out=None) == -1 and call(ws=None) == -1
    assert call(x=ODD) == -1 and call(out=ODD) == -1 and call(ws=ODD) == -1
    assert call(kind=2) == -1
    assert call(size=need - 1) == -3
    for miss in ("w_gate", "w13", "w2", "w13_scales", "w2_scales"):
        assert call(w=_weights(**{miss: None})) == -1, miss
    assert call(w=_weights(w13=0x1008)) == -1
    assert call(w=_weights(expert_layout=moe.LAYOUT_ROWS)) == -1
    assert call(cfg=_cfg(dtype=moe.MXFP4), w=_weights(w13_scales=0x1004),
                size=moe.layer_few_workspace_size(_cfg(dtype=moe.MXFP4))) == -1
    soft = _cfg(scoring=moe.SOFTMAX)
    assert call(cfg=soft, w=_weights(e_bias=0x1000)) == -1
    # MXFP4 belongs to the few-token layer: the others refuse it as before
    assert L.moe_workspace_size(ctypes.byref(_cfg(dtype=moe.MXFP4)), ctypes.byref(n)) == -1


def test_mx4_refusals(L):
    q, d, pk = L.moe_mx4_quantize, L.moe_mx4_dequantize, L.moe_mx4_pack_weights
    assert q(4, 33, FAKE, 0, FAKE, FAKE, None) == -2
    assert q(4, 0, FAKE, 0, FAKE, FAKE, None) == -1 and q(-1, 32, FAKE, 0, FAKE, FAKE, None) == -1
    assert q(4, 32, FAKE, 2, FAKE, FAKE, None) == -1
    assert q(4, 32, None, 0, FAKE, FAKE, None) == -1 and q(4, 32, ODD, 0, FAKE, FAKE, None) == -1
    assert q(4, 32, FAKE, 0, ODD, FAKE, None) == -1 and q(4, 32, FAKE, 0, FAKE, None, None) == -1
    assert d(4, 48, FAKE, FAKE, FAKE, 0, None) == -2
    assert d(4, 64, FAKE, FAKE, FAKE, 5, None) == -1 and d(4, 64, FAKE, FAKE, ODD, 0, None) == -1
    assert q(0, 32, None, 0, None, None, None) == 0 and d(0, 32, None, None, None, 0, None) == 0
    far = P(0x10000000)
    assert pk(2, 100, 128, FAKE, FAKE, far, far, None) == -2
    assert pk(2, 128, 64, FAKE, FAKE, far, far, None) == -2
    assert pk(2, 128, 128, FAKE, FAKE, P(0x1000 + 64), far, None) == -1   # codes overlap
    assert pk(2, 128, 128, FAKE, FAKE, far, P(0x1000), None) == -1        # scales overlap
    assert pk(0, 128, 128, None, None, None, None, None) == 0


def test_mx4_gemm_refusals(L):
    def gemm(groups=2, n=256, k=256, rows=8, a=FAKE, a_s=FAKE, off=FAKE, w=FAKE, w_s=FAKE, c=FAKE, kind=0):
        return L.moe_mx4_grouped_gemm(groups, n, k, rows, a, a_s, off, w, w_s, c, kind, None, None)

    def swiglu(groups=2, inter=256, k=256, rows=8, h=FAKE, h_s=FAKE):
        return L.moe_mx4_grouped_gemm_swiglu(groups, inter, k, rows, FAKE, FAKE, FAKE, FAKE, FAKE, h,
                                             h_s, None, None)
    assert gemm(rows=0, a=None) == 0 and swiglu(rows=0) == 0
    assert gemm(groups=0) == -1 and gemm(rows=-1) == -1 and gemm(kind=3) == -1
    assert gemm(groups=1025) == -2 and gemm(n=200) == -2 and gemm(k=64) == -2
    for name in ("a", "a_s", "off", "w", "w_s", "c"):
        assert gemm(**{name: None}) == -1, name
    for name in ("a", "a_s", "w", "w_s", "c"):
        assert gemm(**{name: ODD}) == -1, name
    assert gemm(c=MIS16) == -1 and swiglu(h=MIS16) == -1   # written 32 bytes at a time
    assert swiglu(inter=192) == -2 and swiglu(inter=0) == -1 and swiglu(inter=2 ** 31 - 1) == -1
    assert swiglu(h=None) == -1 and swiglu(h_s=None) == -1
    assert gemm(groups=1024, n=128 * 1024 * 1024, k=128, rows=2 ** 30) == -2   # tiles beyond 32 bits


def test_norm_refusals(L):
    def norm(T=4, y=FAKE, r=FAKE, gate=None, wp=FAKE, bp=None, wq=FAKE, bq=None, ro=FAKE, xo=FAKE, **kw):
        d = dict(hidden=256, kind=0, y_dtype=0, residual_dtype=0, param_dtype=1, gate_mode=0, eps=1e-6,
                 residual_scale=1.0, branch_scale=1.0)
        d.update(kw)
        return L.moe_block_norm(ctypes.byref(moe.Norm(**d)), T, y, r, gate, wp, bp, wq, bq, ro, xo, None)
    assert norm(T=0) == 0
    assert L.moe_block_norm(None, 4, FAKE, FAKE, None, FAKE, None, FAKE, None, FAKE, FAKE, None) == -1
    assert norm(T=-1) == -1 and norm(hidden=0) == -1 and norm(kind=2) == -1
    assert norm(hidden=260) == -2 and norm(hidden=16392) == -2
    assert norm(eps=-1.0) == -1 and norm(eps=float("nan")) == -1
    assert norm(y_dtype=2) == -1 and norm(residual_dtype=2) == -1 and norm(param_dtype=-1) == -1
    assert norm(gate=FAKE) == -1 and norm(gate_mode=1) == -1 and norm(gate=FAKE, gate_mode=4) == -1
    assert norm(y=None) == -1                              # a post-norm of nothing
    assert norm(y=None, wp=None, gate=FAKE, gate_mode=1) == -1
    assert norm(wp=None, bp=FAKE) == -1 and norm(wq=None, bq=FAKE, xo=None) == -1
    assert norm(wq=None) == -1 and norm(xo=None) == -1     # a pre-norm and its output go together
    assert norm(r=None) == -1 and norm(ro=None, wq=None, xo=None) == -1
    for name in ("y", "r", "wp", "wq", "ro", "xo"):
        assert norm(**{name: ODD}) == -1, name


def test_binding_refuses_wrong_tensors():
    """What the library cannot see: shapes, types and places of tensors."""
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.mx4_quantize(x)                                # not on the GPU
    with pytest.raises(TypeError):
        moe.block._bytes(x, x.shape, "codes")
    with pytest.raises(ValueError):
        moe.block._dense(x, (4, 32), "x")
    with pytest.raises(TypeError):
        moe.block._out_type(x.half())
    b = torch.zeros(64, dtype=torch.bfloat16)
    for bad in (dict(residual=x), dict(residual=x, y=x[:2]), dict(residual=x, residual_out=x.bfloat16()),
                dict(residual=x, x_out=x), dict(residual=x, w_pre=b, gate=b.float()),
                dict(residual=x, gate=b[:3]), dict(residual=x.half()), dict(residual=x.t())):
        with pytest.raises((TypeError, ValueError)):
            moe.block_norm(**bad)
    s = dataclasses.replace(synth.CONFIGS["r1_mini"], dtype="mxfp4")
    assert moe.make_config(s, 4).dtype == moe.BF16         # FewTokenLayer sets its own
