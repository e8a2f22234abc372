"""Products of a few rows with four-bit weights against fp64.

Tolerance: products of a code and an fp16 number are exact, sums are fp32: 32 products in the tensor
cores, then at most 8 blocks, 16 warps and 8 CTAs one after the other, fewer than 64 roundings of
2^-23 at most (the tensor cores truncate): 2^-17 of the sum of the magnitudes.  each x is off by
2^-29 of its row's largest at most: 2^-29 of that times the sum of |w|.  Outputs add half a step: 2^-8 (bf16), 2^-24."""
from __future__ import annotations

import itertools

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from oracle import mx4

from _gpu_common import build_library

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _weights(N, K, kind, group, stype, zeros, g):
    if kind == "mx":
        w = torch.randn(N, K, device="cuda", generator=g) * torch.exp(torch.randn(N, 1, device="cuda", generator=g))
        c, s = moe.mx4_quantize(w)
        return c, s, None, torch.tensor(mx4.dequantize(c.cpu().numpy(), s.cpu().numpy()), device="cuda")
    c = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = (torch.randn(N, K // group, device="cuda", generator=g) * 0.01).to(stype)
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    code = torch.stack([c & 15, c >> 4], -1).flatten(1).double()
    zz = 8.0 if z is None else z.double().repeat_interleave(group, 1)
    return c, s, z, (code - zz) * s.double().repeat_interleave(group, 1)


def _check(x, w64, out):
    ref = x.double() @ w64.t()
    size = x.double().abs() @ w64.abs().t()
    half = 2.0 ** -8 if out.dtype == BF else 2.0 ** -24
    bound = 2.0 ** -17 * size + half * ref.abs() + 2.0 ** -29 * x.double().abs().amax(1, keepdim=True) * w64.abs().sum(1)
    assert bool(((out.double() - ref).abs() <= bound).all()), float(((out.double() - ref).abs() / bound).max())


def _run(T, N, K, kind="mx", group=32, stype=BF, zeros=False, out=BF, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s, z, w64 = _weights(N, K, kind, group, stype, zeros, g)
    x = (torch.randn(T, K, device="cuda", generator=g) * torch.exp(2 * torch.randn(T, 1, device="cuda", generator=g))).bfloat16()
    y = torch.full((T, N), 3.0, dtype=out, device="cuda")
    assert moe.w4_matvec(x, c, s, y, zeros=z) is y
    _check(x, w64, y)
    return x, c, s, z, y


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(16, 32), (1, 64), (17, 128), (100, 160), (1111, 1024), (640, 2048), (257, 2080)])
def test_mx(lib, T, N, K):
    _run(T, N, K, out=F32)


@pytest.mark.parametrize("T,N,K", [(1, 10240, 7168), (16, 7168, 8192), (5, 33, 32768), (16, 48, 32736), (9, 300, 12288)])
@pytest.mark.parametrize("kind", ["mx", "int"])
def test_long_rows(lib, T, N, K, kind):
    _run(T, N, K, kind, 32 if kind == "mx" else 32 if K % 128 else 128)


@pytest.mark.parametrize("group,stype,zeros,out", list(itertools.product((32, 64, 128), (BF, F32), (False, True), (BF, F32))))
@pytest.mark.parametrize("T", [3, 13])
def test_int(lib, group, stype, zeros, out, T):
    _run(T, 333, group * 9, "int", group, stype, zeros, out)
    _run(T, 40, group * 34, "int", group, stype, zeros, out)


def test_many_rows_of_weights(lib):
    """More row tiles than a cluster holds between exchanges."""
    _run(4, 40000, 4224)


def test_rows_do_not_touch_one_another(lib):
    """A NaN or infinity in a row of x, or a block of W, stays in its row or column."""
    x, c, s, _, y = _run(6, 96, 256)
    x[2, 100] = float("nan")
    x[4, 3] = float("inf")
    got = moe.w4_matvec(x, c, s, torch.empty_like(y))
    assert bool(torch.isnan(got[2]).all()) and not bool(torch.isfinite(got[4]).any())
    rest = [0, 1, 3, 5]
    assert torch.equal(got[rest], y[rest])
    s[7, 3] = 255   # a block that is NaN
    c[7, 48:64] = 0
    got = moe.w4_matvec(x[rest].contiguous(), c, s, torch.empty_like(y[rest]))
    assert bool(torch.isnan(got[:, 7]).all())
    keep = [n for n in range(96) if n != 7]
    assert torch.equal(got[:, keep], y[rest][:, keep])


def test_rows_of_zeros_tiny_and_huge_numbers(lib):
    g = torch.Generator(device="cuda").manual_seed(3)
    c, s, _, w64 = _weights(64, 512, "mx", 32, None, False, g)
    x = torch.randn(5, 512, device="cuda", generator=g)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e30
    x[3, ::2] *= 1e-9
    x[4] *= 1e-38   # and the smallest of all: subnormal numbers
    x = x.bfloat16()
    y = torch.empty(5, 64, device="cuda")
    moe.w4_matvec(x, c, s, y)
    assert not bool(y[0].any())
    _check(x, w64, y)


def test_same_bits_each_time_and_on_another_stream(lib):
    x, c, s, z, y = _run(11, 500, 7168, "int", 64, F32, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(y) for _ in range(4)]
    for o in outs[:2]:
        moe.w4_matvec(x, c, s, o, zeros=z)
    for o in outs[2:]:
        moe.w4_matvec(x, c, s, o, zeros=z, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)


def test_no_rows(lib):
    moe.w4_matvec(torch.empty(0, 64, dtype=BF, device="cuda"), torch.zeros(8, 32, dtype=torch.uint8, device="cuda"),
                  torch.zeros(8, 2, dtype=torch.uint8, device="cuda"), torch.empty(0, 8, device="cuda"))
