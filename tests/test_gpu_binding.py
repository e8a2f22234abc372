"""What the binding refuses of the tensors of a call: each of these would be read or written out of
its bounds, or as another type."""
from __future__ import annotations

import dataclasses

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
import synth

from _gpu_common import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _empty(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_product_tensors(lib):
    G, N, K, R = 3, 256, 384, 10
    good = dict(a=_empty(R, K // 2), a_scales=_empty(R, K // 32), w=_empty(G, N, K // 2),
                w_scales=_empty(G, N, K // 32), c=_empty(R, N, dtype=torch.float32),
                expert_offsets=torch.tensor([0, 2, 2, R], dtype=torch.int32, device="cuda"),
                status=_empty(1, dtype=torch.int32))

    def call(kind=moe.OUT_F32, rows=R, **kw):
        v = {**good, **kw}
        moe.mx4_grouped_gemm(G, N, K, rows, v["a"], v["a_scales"], v["expert_offsets"], v["w"],
                             v["w_scales"], v["c"], kind, v["status"])
    call()
    call(a=_empty(R + 3, K // 2), c=_empty(R + 1, N, dtype=torch.float32))   # more rows than used
    call(status=None, expert_offsets=good["expert_offsets"].data_ptr())
    call(c=good["c"].bfloat16(), kind=moe.OUT_BF16)
    for name, bad in (
            ("a", good["a"][:-1]), ("a", good["a"].int()), ("a", good["a"].cpu()),
            ("a", _empty(R, K)), ("a", _empty(K // 2, R).t()), ("a_scales", good["a_scales"][:-1]),
            ("a_scales", _empty(R, K // 16)), ("w", good["w"][:-1]), ("w", _empty(G * 2, N // 2, K // 2)),
            ("w_scales", good["w_scales"][1:]), ("w_scales", _empty(G, N, K // 32, dtype=torch.int32)),
            ("c", good["c"][:-1]), ("c", good["c"].bfloat16()), ("c", good["c"].half()),
            ("expert_offsets", good["expert_offsets"][:-1]), ("expert_offsets", good["expert_offsets"].long()),
            ("status", _empty(1))):
        with pytest.raises((TypeError, ValueError)):
            call(**{name: bad})
    with pytest.raises((TypeError, ValueError)):
        call(kind=moe.OUT_BF16)
    with pytest.raises(moe.MoEError):
        call(kind=9)
    with pytest.raises(moe.MoEError):
        call(a=None)
    call(rows=0, a=None)


def test_swiglu_tensors(lib):
    G, I, K, R = 2, 128, 256, 5
    off = torch.tensor([0, 2, R], dtype=torch.int32, device="cuda")
    good = dict(h=_empty(R, I // 2), h_scales=_empty(R, I // 32), w13=_empty(G, 2 * I, K // 2))

    def call(**kw):
        v = {**good, **kw}
        moe.mx4_grouped_gemm_swiglu(G, I, K, R, _empty(R, K // 2), _empty(R, K // 32), off, v["w13"],
                                    _empty(G, 2 * I, K // 32), v["h"], v["h_scales"])
    call()
    for name, bad in (("h", _empty(R, I)), ("h", good["h"][1:]), ("h_scales", good["h_scales"].int()),
                      ("h_scales", good["h_scales"][:-1]), ("w13", good["w13"][:, :I].contiguous())):
        with pytest.raises((TypeError, ValueError)):
            call(**{name: bad})


def _layer(dtype="bf16", T=20, few=True):
    shape = synth.MoEShape("io", tokens=T, hidden=256, inter=128, num_experts=4, num_shared=1, top_k=2,
                           dtype="bf16")
    w = synth.make_inputs(shape, device="cuda")
    if dtype == "mxfp4":
        for key in ("w13", "w2"):
            w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
        shape = dataclasses.replace(shape, dtype=dtype)
    return (moe.FewTokenLayer(shape, w) if few else moe.Mx4MoELayer(shape, w, T)), w["x"]


@pytest.mark.parametrize("kind,T", [("few", 3), ("mxfp4", 3), ("mxfp4", 20)])
def test_layer_input_and_output(lib, kind, T):
    layer, x = _layer("mxfp4" if kind == "mxfp4" else "bf16", few=kind == "few")
    x = x[:T].contiguous()
    f32, bf = _empty(T, 256, dtype=torch.float32), _empty(T, 256, dtype=torch.bfloat16)
    assert layer.forward(x, f32) is f32 and layer.forward(x, bf) is bf      # out's own type
    assert torch.equal(f32.bfloat16(), bf)
    layer.forward(x, bf, moe.OUT_BF16)
    guarded = torch.full((T + 2, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    layer.forward(x, guarded[1:-1])
    assert torch.equal(guarded[1:-1], bf) and bool((guarded[0] == 7).all() & (guarded[-1] == 7).all())
    for bad in (dict(x=x.float()), dict(x=x.half()), dict(x=x[:, :128].contiguous()), dict(x=x.cpu()),
                dict(x=torch.cat([x, x], 1)[:, ::2]), dict(out=f32[:-1]), dict(out=f32.half()),
                dict(out=f32[:, :128].contiguous()), dict(out=_empty(T, 512, dtype=torch.float32)[:, :256]),
                dict(out=bf, out_dtype=moe.OUT_F32), dict(out=f32, out_dtype=moe.OUT_BF16),
                dict(x=x.reshape(-1)), dict(out=f32.cpu())):
        with pytest.raises((TypeError, ValueError)):
            layer.forward(**{"x": x, "out": f32, **bad})
    if kind == "few":
        with pytest.raises(ValueError):
            layer.forward(x, f32, T=T + 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
def test_weights_of_the_few_token_layer(lib, dtype):
    shape = synth.MoEShape("w", tokens=4, hidden=256, inter=128, num_experts=4, num_shared=1, top_k=2,
                           dtype="bf16" if dtype == "mxfp4" else dtype, scoring="sigmoid", bias_std=0.1)
    w = synth.make_inputs(shape, device="cuda")
    if dtype == "mxfp4":
        for key in ("w13", "w2"):
            w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
    shape = dataclasses.replace(shape, dtype=dtype)
    w["logit_offset"] = _empty(4, dtype=torch.float32)
    moe.FewTokenLayer(shape, w, log2phys=[3, 2, 1, 0])
    for key, t in w.items():
        if key == "x" or t is None:
            continue
        for bad in (t[:-1], t.double(), t.cpu()):
            with pytest.raises((TypeError, ValueError)):
                moe.FewTokenLayer(shape, dict(w, **{key: bad}))
    for table in ([0, 1, 2], [0] * 5):
        with pytest.raises(ValueError):
            moe.FewTokenLayer(shape, w, log2phys=table)


def test_a_layer_of_other_sizes_or_another_table(lib):
    shape = synth.MoEShape("w", tokens=4, hidden=256, inter=256, num_experts=4, num_shared=1, top_k=2,
                           dtype="fp8")
    big = moe.MoELayer(shape, synth.make_inputs(shape, device="cuda"), log2phys=[1, 0, 3, 2])
    moe.FewTokenLayer(shape, big)
    with pytest.raises(ValueError):
        moe.FewTokenLayer(shape, big, log2phys=[0, 1, 2, 3])
    for change in (dict(hidden=512), dict(inter=128), dict(num_experts=8), dict(num_shared=0),
                   dict(dtype="bf16"), dict(dtype="mxfp4")):
        with pytest.raises(ValueError):
            moe.FewTokenLayer(dataclasses.replace(shape, **change), big)
