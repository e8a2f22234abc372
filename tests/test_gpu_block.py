"""The operators together, as a decoder's MoE block runs them: pre-norm, layer, post-norm with gate
and residual scale, for every expert type and on both sides of the few-token bound.

Each step is compared with fp64 on what the step before it stored: the norms within half a bf16
unit, the layer (its definition: x and h rounded to the experts' type) within 2e-2 of its output in
the Euclidean norm -- half a bf16 unit is 1.7e-3 of that, and a value of h next to a rounding
boundary may take the other code, one of which weighs up to 1e-2 in a single token."""
from __future__ import annotations

import dataclasses
import os
import subprocess
import sys

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
import synth
from oracle import mx4

from _gpu_common import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _norm64(v, w):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w.double()


def _rounded(shape, v):
    """v fp64 by the values that its form in the experts' type stands for."""
    if shape.dtype == "bf16":
        return v.bfloat16().double()
    if shape.dtype == "mxfp4":
        return torch.tensor(mx4.dequantize(*mx4.quantize(v.cpu().numpy())), device="cuda")
    b = v.float().view(v.shape[0], -1, 128)
    s = (b.abs().amax(-1, keepdim=True) / torch.full((1,), 448.0, device="cuda")).clamp(min=1e-30)
    return ((b / s).to(torch.float8_e4m3fn).double() * s.double()).view(v.shape)


def _layer64(shape, w, x):
    """The layer in fp64 on bf16 x."""
    T = x.shape[0]
    cfg = moe.make_config(dataclasses.replace(shape, dtype="bf16"), T)
    logits = torch.empty(T, shape.num_experts, device="cuda")
    ids = torch.empty(T, shape.top_k, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, shape.top_k, device="cuda")
    moe.route(cfg, T, x, w["wg"], w.get("e_bias"), None, None, logits, ids, tw)
    xq = _rounded(shape, x.double())
    out = torch.zeros(T, shape.hidden, dtype=torch.float64, device="cuda")
    dense = torch.zeros(T, shape.groups, dtype=torch.float64, device="cuda")
    dense.scatter_(1, ids.long(), tw.double())
    dense[:, shape.num_experts:] = 1.0
    for g in range(shape.groups):
        rows = dense[:, g].nonzero()[:, 0]
        if not len(rows):
            continue
        v13, v2 = (_values(shape, w, key, g) for key in ("w13", "w2"))
        o = xq[rows] @ v13.t()
        h = o[:, :shape.inter] / (1 + torch.exp(-o[:, :shape.inter])) * o[:, shape.inter:]
        h = _rounded(shape, h)
        out[rows] += dense[rows, g, None] * (h @ v2.t())
    return out


def _values(shape, w, key, g):
    if shape.dtype == "bf16":
        return w[key][g].double()
    if shape.dtype == "fp8":
        s = w[key + "_s"][g].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return w[key][g].view(torch.float8_e4m3fn).double() * s
    return moe.mx4_dequantize(w[key][g], w[key + "_s"][g]).double()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T", [1, 16, 17, 70])
def test_block(lib, dtype, T):
    shape = synth.MoEShape("blk", tokens=T, hidden=512, inter=384, num_experts=16, num_shared=1,
                           top_k=4, dtype="bf16" if dtype == "mxfp4" else dtype)
    w = synth.make_inputs(shape, seed=T, device="cuda")
    if dtype == "mxfp4":
        for key in ("w13", "w2"):
            w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
        shape = dataclasses.replace(shape, dtype="mxfp4")
        layer, few = moe.Mx4MoELayer(shape, w, 128), None
    else:
        layer = moe.MoELayer(shape, w, max_tokens=128)
        few = moe.FewTokenLayer(shape, layer)
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w_pre, w_post = (1 + 0.1 * rnd(512)).bfloat16(), (1 + 0.1 * rnd(512)).bfloat16()
    w_next, gate = (1 + 0.1 * rnd(512)).bfloat16(), rnd(512).bfloat16()
    blk = moe.MoEBlock(layer, w_pre, w_post, gate, residual_scale=0.9, branch_scale=0.5, few=few)
    r0 = rnd(T, 512) * 2
    r, x = r0.clone(), torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    blk.pre(r, x)
    half = lambda v: torch.exp2(torch.frexp(v)[1].double() - 9)  # noqa: E731
    ref = _norm64(r0.double(), w_pre)
    assert bool(((x.double() - ref).abs() <= half(ref) + 1e-5).all())
    xin, x_next = x.clone(), torch.empty_like(x)
    blk.forward(r, x, y, w_next=w_next, x_next=x_next)
    ref = _layer64(shape, w, xin)
    assert float((y.double() - ref).norm()) <= 2e-2 * float(ref.norm())
    rr = 0.9 * r0.double() + 0.5 * gate.double() * _norm64(y.double(), w_post)
    assert float((r.double() - rr).abs().max()) <= 2e-5 * float(rr.abs().max())
    nx = _norm64(rr, w_next)
    assert bool(((x_next.double() - nx).abs() <= half(nx) + 1e-4).all())
    assert (few if few is not None and T <= 16 else layer).status() == 0


def test_paths_of_the_mxfp4_layer_agree(lib):
    """The same tokens through the few-token kernels and through the products: h may differ by a
    code where it lies on a rounding boundary, so the outputs agree to a small part of their size."""
    shape = synth.MoEShape("two", tokens=40, hidden=1024, inter=512, num_experts=16, num_shared=1,
                           top_k=4)
    w = synth.make_inputs(shape, seed=1, device="cuda")
    for key in ("w13", "w2"):
        w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
    layer = moe.Mx4MoELayer(dataclasses.replace(shape, dtype="mxfp4"), w, 40)
    big = torch.empty(40, 1024, device="cuda")
    layer.forward(w["x"], big)
    few = torch.cat([layer.forward(w["x"][i:i + 8].contiguous(), torch.empty(8, 1024, device="cuda"))
                     for i in range(0, 40, 8)])
    assert float((big - few).square().mean().sqrt()) <= 2e-3 * float(big.square().mean().sqrt())
    assert layer.status() == 0


def test_example(lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "moe_block.py"), "--hidden",
                        "512", "--inter", "256", "--experts", "16", "--top-k", "4", "--prompt", "40"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "decode step" in r.stdout
