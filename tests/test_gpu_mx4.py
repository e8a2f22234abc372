"""MXFP4 quantisation, its inverse and the weight packing: every bit against the oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from oracle import mx4

from _gpu_common import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _rows(rows, cols, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))
    return v.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (37, 1024), (129, 7168), (2050, 416)])
def test_codes_and_scales_equal_the_oracle(lib, rows, cols, dtype):
    v = _rows(rows, cols, rows + cols, dtype)
    codes, scales = moe.mx4_quantize(v.cuda())
    c, s = mx4.quantize(v.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    for out in (torch.float32, torch.bfloat16):
        got = moe.mx4_dequantize(codes, scales, torch.empty(rows, cols, dtype=out, device="cuda"))
        assert np.array_equal(got.cpu().double().numpy(), mx4.dequantize(c, s))


def test_edges(lib):
    """Zeros, ties, subnormal numbers, the largest numbers, infinities and NaN; the blocks beside
    a bad one are untouched by it."""
    blocks = torch.zeros(12, 32)
    blocks[1, :10] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0])
    blocks[2, 3] = 2.0 ** -149
    blocks[3, :3] = torch.tensor([2.0 ** -127, -(2.0 ** -128), 2.0 ** -140])
    blocks[4, :2] = torch.tensor([torch.finfo(torch.float32).max, -1e38])
    blocks[5, 31] = float("inf")
    blocks[6, 0] = float("nan")
    blocks[7] = 1.0
    blocks[8, 5], blocks[8, 6] = float("-inf"), float("nan")
    blocks[9] = -0.0
    blocks[10, :4] = torch.tensor([7.0, 6.999, 5.001, 4.999])
    blocks[11] = torch.linspace(-1, 1, 32)
    v = blocks.reshape(3, 128)
    codes, scales = moe.mx4_quantize(v.cuda())
    c, s = mx4.quantize(v.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    got = moe.mx4_dequantize(codes, scales, torch.empty(3, 128, device="cuda")).cpu().numpy()
    assert np.array_equal(got, mx4.dequantize(c, s).astype(np.float32), equal_nan=True)


def test_every_code_and_scale_reads_back(lib):
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(8).reshape(8, 256)
    codes = torch.arange(256, dtype=torch.uint8).repeat(8 * 256 * 16 // 256).reshape(8, 4096)
    got = moe.mx4_dequantize(codes.cuda(), scales.cuda(), torch.empty(8, 8192, device="cuda"))
    # an fp32 number from 2^128 on overflows (6 * 2^126 and the like cannot be stored)
    with np.errstate(over="ignore"):
        ref = mx4.dequantize(codes.numpy(), scales.numpy()).astype(np.float32)
    assert np.array_equal(got.cpu().numpy(), ref, equal_nan=True)


def test_more_than_two_to_the_31_elements(lib):
    rows, cols = 70000, 32768   # 2.3e9 elements
    v = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    v.fill_(1.0)
    v[-1] = torch.arange(cols, device="cuda") % 7
    codes, scales = moe.mx4_quantize(v)
    out = moe.mx4_dequantize(codes, scales)
    assert torch.equal(out[-1].float().cpu().double(), torch.tensor(
        mx4.dequantize(*mx4.quantize(v[-1:].cpu().double().numpy())))[0])
    assert bool((out[:-1] == 1.0).all())


def test_no_rows(lib):
    codes, scales = moe.mx4_quantize(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert moe.mx4_dequantize(codes, scales).shape == (0, 64)


@pytest.mark.parametrize("G,N,K", [(1, 128, 128), (3, 256, 384), (2, 128, 1408)])
def test_pack_is_the_tile_permutation(lib, G, N, K):
    g = torch.Generator().manual_seed(G)
    codes = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, generator=g)
    scales = torch.randint(0, 256, (G, N, K // 32), dtype=torch.uint8, generator=g)
    w, ws = moe.pack_mx4_weights(codes.cuda(), scales.cuda())
    t = codes.view(G, N // 128, 128, K // 128, 4, 16).permute(0, 1, 3, 2, 4, 5)
    r, c = torch.arange(128)[:, None], torch.arange(4)[None, :]
    t = t[:, :, :, r, c ^ ((r // 2) % 4), :]
    assert torch.equal(w.cpu().reshape(-1), t.reshape(-1))
    u = scales.view(G, N // 128, 4, 32, K // 128, 4).permute(0, 1, 4, 3, 2, 5)
    assert torch.equal(ws.cpu().reshape(-1), u.reshape(-1))


def test_another_stream(lib):
    """Work is enqueued on the given stream: its own input is written there first."""
    s = torch.cuda.Stream()
    v = _rows(512, 7168, 1, torch.float32)
    with torch.cuda.stream(s):
        d = v.cuda(non_blocking=True) * 1.0
        codes, scales = moe.mx4_quantize(d)
    s.synchronize()
    c, b = mx4.quantize(v.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), b)
