"""The norms around a block against their formula in fp64.

Tolerance: everything is fp32 with a handful of roundings a value and sums over at most 16384
terms in a tree of short chains, so a value is within 1e-5 of its own size plus that of the
terms it is the sum of; bf16 outputs add half a unit in the last place (eight significant bits: 2^(e-9) for a value in
[2^(e-1), 2^e))."""
from __future__ import annotations

import itertools

import pytest
import torch

import moe_expert_layer_07_gb300 as moe

from _gpu_common import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _norm64(v, kind, eps, w, b):
    if kind == moe.NORM_LAYER:
        v = v - v.mean(-1, keepdim=True)
    n = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w.double()
    return n if b is None else n + b.double()


def _reference(a, alpha, beta, eps, kind):
    r = alpha * a["residual"].double()
    size = r.abs()
    if a.get("y") is not None:
        n = a["y"].double()
        if a.get("w_post") is not None:
            n = _norm64(n, kind, eps, a["w_post"], a.get("b_post"))
        if a.get("gate") is not None:
            g = a["gate"].double()
            n = n * (g[:, None] if g.dim() == 1 and g.shape[0] != n.shape[1] else g)
        r = r + beta * n
        size = size + abs(beta) * n.abs()
    x = _norm64(r, kind, eps, a["w_pre"], a.get("b_pre")) if a.get("w_pre") is not None else None
    return r, x, size


def _close(got, ref, slack, dtype):
    bound = 1e-5 * (ref.abs() + slack)
    if dtype == torch.bfloat16:
        bound = bound + torch.exp2(torch.frexp(ref)[1].double() - 9)
    assert bool(((got.double() - ref).abs() <= bound).all()), \
        float(((got.double() - ref).abs() / bound).max())


def _inputs(T, H, y, res, param, bias, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale + shift).to(dtype)

    a = {"residual": r(T, H, dtype=res, scale=3.0, shift=0.5)}
    if y is not None:
        a["y"] = r(T, H, dtype=y, scale=0.5, shift=0.2)
        a["w_post"] = r(H, dtype=param, scale=0.1, shift=1.0)
        a["b_post"] = r(H, dtype=param, scale=0.1) if bias else None
        if gate:
            a["gate"] = r(*{"feature": (H,), "token": (T,), "full": (T, H)}[gate], dtype=param)
    a["w_pre"] = r(H, dtype=param, scale=0.1, shift=1.0)
    a["b_pre"] = r(H, dtype=param, scale=0.1) if bias else None
    return a


def _run(a, alpha=0.8, beta=0.4, eps=1e-6, kind=0):
    out = torch.empty_like(a["residual"])
    x = torch.empty(a["residual"].shape, dtype=torch.bfloat16, device="cuda")
    moe.block_norm(**a, residual_out=out, x_out=x, residual_scale=alpha, branch_scale=beta, eps=eps,
                   kind=kind)
    r64, x64, size = _reference(a, alpha, beta, eps, kind)
    _close(out, r64, size, out.dtype)
    # a normed value also carries the error of its mean and of its row's inverse size
    scale = x64.abs().mean(-1, keepdim=True) * 4
    _close(x, x64, scale + size * (x64.abs().mean(-1, keepdim=True) /
                                   r64.abs().mean(-1, keepdim=True).clamp(min=1e-30)), x.dtype)
    return out, x


F32, BF = torch.float32, torch.bfloat16


@pytest.mark.parametrize("y,res,param", list(itertools.product((F32, BF), repeat=3)))
@pytest.mark.parametrize("kind", [0, 1])
def test_types(lib, y, res, param, kind):
    _run(_inputs(5, 1024, y, res, param, kind == 1, "feature"), kind=kind)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (2, 248), (3, 264), (7, 2048), (33, 1416),
                                 (2, 8192), (2, 8200), (3, 16384), (1000, 7168)])
@pytest.mark.parametrize("kind", [0, 1])
def test_sizes(lib, T, H, kind):
    _run(_inputs(T, H, F32, BF, BF, False, None), kind=kind)


@pytest.mark.parametrize("gate", [None, "feature", "token", "full"])
@pytest.mark.parametrize("T", [1, 6])
def test_gates(lib, gate, T):
    _run(_inputs(T, 512, BF, F32, BF, True, gate), kind=1)


def test_one_token_gate_of_one_feature_row(lib):
    """[H] and [T, H] agree for one token."""
    a = _inputs(1, 256, F32, F32, F32, False, "feature")
    out, x = _run(a)
    b = dict(a, gate=a["gate"].reshape(1, 256))
    out2, x2 = _run(b)
    assert torch.equal(out, out2) and torch.equal(x, x2)


def test_pre_norm_alone_and_post_norm_alone(lib):
    a = _inputs(4, 768, None, BF, BF, False, None)
    _run(a)   # no branch
    b = _inputs(4, 768, F32, F32, BF, False, None)
    out = torch.empty_like(b["residual"])
    moe.block_norm(b["residual"], y=b["y"], residual_out=out, w_post=b["w_post"])
    r64, _, size = _reference({**b, "w_pre": None}, 1.0, 1.0, 1e-6, 0)
    _close(out, r64, size, F32)
    # neither norm: the scaled sum
    moe.block_norm(b["residual"], y=b["y"], residual_out=out, residual_scale=0.5, branch_scale=2.0)
    ref = 0.5 * b["residual"].double() + 2.0 * b["y"].double()
    _close(out, ref, ref.abs(), F32)


def test_residual_in_place(lib):
    a = _inputs(9, 2048, BF, BF, BF, False, "full")
    want, wx = _run(a)
    res = a["residual"].clone()
    x = torch.empty_like(wx)
    moe.block_norm(**{**a, "residual": res}, residual_out=res, x_out=x, residual_scale=0.8,
                   branch_scale=0.4)
    assert torch.equal(res, want) and torch.equal(x, wx)


def test_rows_of_zeros_large_means_and_non_finite_rows(lib):
    a = _inputs(6, 1024, F32, F32, F32, False, None)
    a["y"][0] = 0.0
    a["residual"][0] = 0.0
    a["y"][1] = 1000.0 + torch.linspace(-1, 1, 1024, device="cuda")   # a mean far above the spread
    a["y"][2, 7] = float("inf")
    a["y"][3, 9] = float("nan")
    out, x = torch.empty_like(a["residual"]), torch.empty(6, 1024, dtype=BF, device="cuda")
    moe.block_norm(**a, residual_out=out, x_out=x, kind=moe.NORM_LAYER)
    assert not out[0].any() and not x[0].any()
    r64, _, size = _reference(a, 1.0, 1.0, 1e-6, moe.NORM_LAYER)
    # the mean of values near 1000 rounds at 2^-24 * 1000, of a spread of 0.58
    assert float((out[1].double() - r64[1]).abs().max()) < 1e-3
    assert bool(torch.isnan(out[2:4]).any(-1).all()) and bool(torch.isnan(x[2:4]).all())
    _close(out[4:], r64[4:], size[4:], F32)   # their neighbours are untouched
    assert bool(torch.isfinite(x[4:]).all())


def test_no_rows(lib):
    e = torch.empty(0, 64, device="cuda")
    moe.block_norm(e, residual_out=e)
