"""The kernel variants that only large calls take: norms of many rows, MXFP4 quantisation and
read-back with four chunks a thread.  MXFP4 is compared bit for bit.

Norms: everything is fp32 with a handful of roundings a value and sums over at most 16384 terms in
trees of short chains, so a value is within 1e-5 of the sizes of all terms it is the sum of, added up
(the rule of test_gpu_norm.py, which leaves out the terms inside a norm: with millions of values some
cancel there).  bf16 outputs add half a unit in the last place."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from oracle import mx4

from _gpu_common import build_library
from test_gpu_norm import BF, F32, _inputs

pytestmark = pytest.mark.gpu


def _normed(v, size, kind, w, b):
    """norm(v) w + b in fp64, and the size of its terms where v's have `size`."""
    mean = v.mean(-1, keepdim=True) if kind == moe.NORM_LAYER else torch.zeros_like(v[:, :1])
    inv = 1 / torch.sqrt((v - mean).square().mean(-1, keepdim=True) + 1e-6)
    n, s = (v - mean) * inv * w.double(), (size + mean.abs()) * inv * w.double().abs()
    return (n, s) if b is None else (n + b.double(), s + b.double().abs())


def _within(got, ref, size):
    bound = 1e-5 * size
    if got.dtype == BF:
        bound = bound + torch.exp2(torch.frexp(ref)[1].double() - 9)
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


def _run(a, kind=moe.NORM_RMS):
    out = torch.empty_like(a["residual"])
    x = torch.empty(out.shape, dtype=BF, device="cuda")
    moe.block_norm(**a, residual_out=out, x_out=x, residual_scale=0.8, branch_scale=0.4, kind=kind)
    r = 0.8 * a["residual"].double()
    size = r.abs()
    if a.get("y") is not None:
        n = a["y"].double()
        n, s = _normed(n, n.abs(), kind, a["w_post"], a.get("b_post"))
        if a.get("gate") is not None:
            g = a["gate"].double()
            g = g[:, None] if g.shape == n.shape[:1] else g
            n, s = n * g, s * g.abs()
        r, size = r + 0.4 * n, size + 0.4 * s
    _within(out, r, size)
    _within(x, *_normed(r, size, kind, a["w_pre"], a.get("b_pre")))
    return out, x


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


# one, two, four and eight chunks of a row to a thread; 248 and 256 columns: eight rows to a CTA, the
# last one not full; sizes that leave threads without a chunk
@pytest.mark.parametrize("T,H", [(700, 7168), (700, 4104), (400, 8192), (700, 1024), (700, 520), (700, 4096),
                                 (2051, 248), (2051, 256), (1003, 512), (401, 8200), (401, 16384)])
@pytest.mark.parametrize("y,res", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("kind", [0, 1])
def test_norms_of_many_rows(lib, T, H, y, res, kind):
    for gate in (None, "feature", "token", "full"):
        _run(_inputs(T, H, y, res, BF if kind else F32, kind == 1, gate, seed=H + kind), kind=kind)


@pytest.mark.parametrize("T,H", [(700, 7168), (2051, 248)])
def test_many_rows_without_a_branch_and_in_place(lib, T, H):
    a = _inputs(T, H, None, BF, BF, False, None)
    _run(a)
    a = _inputs(T, H, BF, BF, BF, False, "full")
    want, wx = _run(a)
    x = torch.empty_like(wx)
    moe.block_norm(**a, residual_out=a["residual"], x_out=x, residual_scale=0.8, branch_scale=0.4)
    assert torch.equal(a["residual"], want) and torch.equal(x, wx)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1531, 3061])   # one round of the loop, and two
def test_mxfp4_of_many_rows(lib, rows, dtype):
    """Chunk counts that four chunks a thread do not divide."""
    cols = 7200
    assert rows * cols // 8 % 1024
    g = torch.Generator().manual_seed(rows)
    v = (torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))).to(dtype)
    v[7, 40], v[-1, -1] = float("inf"), float("nan")
    guard = torch.full((rows * cols // 2 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    codes = guard[32:-32].view(rows, cols // 2)
    codes, scales = moe.mx4_quantize(v.cuda(), codes)
    c, s = mx4.quantize(v.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), c)
    assert bool((guard[:32] == 0xA5).all()) and bool((guard[-32:] == 0xA5).all())
    ref = mx4.dequantize(c, s).astype(np.float32)
    for out in (torch.float32, torch.bfloat16):
        whole = torch.full((rows * cols + 64,), 3.0, dtype=out, device="cuda")
        got = moe.mx4_dequantize(codes, scales, whole[32:-32].view(rows, cols))
        assert np.array_equal(got.float().cpu().numpy(), ref, equal_nan=True)   # exact in bf16 too
        assert bool((whole[:32] == 3.0).all()) and bool((whole[-32:] == 3.0).all())
