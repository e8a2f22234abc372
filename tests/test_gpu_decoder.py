"""The operators of attention together, as a decoder's attention block runs them: tables, projection,
norm and rotation with the cache's write, attention, projection, norm.

Each step is compared with fp64 on what the step before it stored: projections of up to 16 rows within
half a bf16 step (2^-8) and 2^-17 of the sum of magnitudes; of more rows the same on x's own MXFP4 form; the
rest within the tolerances of its own tests, summed up: 2^-7 of the mean magnitude of the values."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from oracle import mx4

from _gpu_common import build_library

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _rounded(v):
    return torch.tensor(mx4.dequantize(*mx4.quantize(v.double().cpu().numpy())), device="cuda")


def _projection(x, w, got):
    w64 = torch.tensor(mx4.dequantize(w[0].cpu().numpy(), w[1].cpu().numpy()), device="cuda")
    x64 = x.double() if x.shape[0] <= 16 else _rounded(x)
    ref, size = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -17 * size + 2.0 ** -29 * x64.abs().amax() * w64.abs().sum(1)
    assert bool(((got.double() - ref).abs() <= bound).all())


def _make(requests, max_rows, max_len, window=0, Hq=8, Hk=2, D=128, hidden=384, page=16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w = [moe.mx4_quantize((r(n, k) * k ** -0.5).bfloat16())
         for n, k in (((Hq + 2 * Hk) * D, hidden), (hidden, Hq * D))]
    max_pages = -(-max_len // page)
    cache = moe.Cache4(requests * max_pages + 2, page, Hk, D)
    cache.codes.fill_(0x77), cache.scales.fill_(255)   # nothing that was not written may be seen
    head = (1 + 0.1 * r(2, D)).bfloat16()
    block = moe.AttentionBlock(cache, Hq, hidden, w[0], w[1], moe.rope_table(max_len, D), requests, max_rows,
                               max_pages, max_q=max_len, max_len=max_len, w_q=head[0], w_k=head[1],
                               w_pre=(1 + 0.1 * r(hidden)).bfloat16(), w_post=(1 + 0.1 * r(hidden)).bfloat16(),
                               gate=r(hidden).bfloat16(), residual_scale=0.9, branch_scale=0.5, window=window)
    return block, moe.PageTables(cache, requests, max_pages, max_rows), r


def _step(block, tables, r, new, pad, history, window, check=True):
    """One step of `new` tokens for each request; history[b]: the cached (k, v) of request b so far."""
    T, H = sum(new) + pad, block.hidden
    Hq, Hk, D = block.q_heads, block.cache.kv_heads, block.cache.dim
    residual = r(T, H)
    x, y = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    tables.step(torch.tensor(new, dtype=I32, device="cuda"))
    block.pre(residual, x)
    x0, r0 = x.clone(), residual.clone()
    w_next = (1 + 0.1 * r(H)).bfloat16()
    block.forward(residual, x, y, tables, w_next=w_next, x_next=x)
    n = sum(new)
    qkv, o = block.qkv[:n], block.q[:n]
    _projection(x0, block.weights[0], block.qkv[:T])
    # keys and values of the new tokens as the cache holds them
    k, v = torch.empty(n, Hk, D, dtype=BF, device="cuda"), torch.empty(n, Hk, D, dtype=BF, device="cuda")
    moe.cache_read(block.cache, tables.slots[:n].contiguous(), k, v)
    z = qkv.double().reshape(n, Hq + 2 * Hk, D)
    assert torch.equal(v.double(), _rounded(z[:, Hq + Hk:]))
    pos = tables.positions[:n].long()
    cs = block.cos_sin.double()[pos][:, None]
    cos, sin = cs[..., :D // 2], cs[..., D // 2:]

    def turned(t, w):
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w.double()
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    kk = _rounded(turned(z[:, Hq:Hq + Hk], block.w_k))
    assert float((kk != k.double()).double().mean()) < 1e-3
    q = turned(z[:, :Hq], block.w_q)
    at = 0
    for b, m in enumerate(new):
        history[b] = (torch.cat([history[b][0], k[at:at + m].double()]), torch.cat([history[b][1], v[at:at + m].double()]))
        kb, vb = history[b]
        L = kb.shape[0]
        assert int(tables.lengths[b]) == L
        if m:
            s = torch.einsum("nhgd,lhd->nhgl", q[at:at + m].reshape(m, Hk, Hq // Hk, D), kb) * D ** -0.5
            p, j = torch.arange(L - m, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
            seen = (j <= p) & ((j > p - window) if window else True)
            w = torch.softmax(s.masked_fill(~seen[:, None, None], float("-inf")), -1)
            ref = torch.einsum("nhgl,lhd->nhgd", w, vb).reshape(m, Hq, D)
            mean = torch.einsum("nhgl,lhd->nhgd", w, vb.abs()).reshape(m, Hq, D)
            # q was rounded to bf16 before the scores: they move by up to 2^-8 of their terms
            spread = 1 + float((s.abs().amax()))
            assert bool(((o[at:at + m].double() - ref).abs() <= 2.0 ** -7 * spread * mean + 1e-6).all())
        at += m
    _projection(block.q[:T].view(T, -1)[:n] if T <= 16 else block.q[:T].view(T, -1), block.weights[1], y[:n] if T <= 16 else y)
    norm = y.double()[:n]
    norm = norm / torch.sqrt((norm * norm).mean(-1, keepdim=True) + 1e-6) * block.w_post.double()
    want = 0.9 * r0.double()[:n] + 0.5 * block.gate.double() * norm
    assert bool(((residual[:n].double() - want).abs() <= 1e-5 * (1 + want.abs() + norm.abs())).all())
    xn = want / torch.sqrt((want * want).mean(-1, keepdim=True) + 1e-6) * w_next.double()
    assert bool(((x[:n].double() - xn).abs() <= 2.0 ** -8 * xn.abs() + 1e-4).all())


@pytest.mark.parametrize("window", [0, 20])
def test_steps(lib, window):
    """Prompts, a mixed step, decode steps with waiting requests and padding rows."""
    block, tables, r = _make(4, 90, 160, window)
    none = (torch.zeros(0, 2, 128, dtype=torch.float64, device="cuda"),) * 2
    history = [none] * 4
    for new, pad in (([5, 1, 0, 3], 0), ([40, 1, 17, 0], 7), ([1, 1, 1, 1], 3), ([1, 0, 1, 1], 0), ([2, 70, 1, 4], 2),
                     ([1, 1, 1, 1], 12)):
        _step(block, tables, r, new, pad, history, window)
    assert int(tables.status) == 0 and block.status() == 0
    # request 1 ends; its pages serve another
    tables.release(1, history[1][0].shape[0])
    history[1] = none
    for new in ([1, 33, 1, 1], [1, 1, 1, 1]):
        _step(block, tables, r, new, 0, history, window)
    assert int(tables.status) == 0 and block.status() == 0


def test_two_blocks_and_streams(lib):
    """Two blocks, each on a stream of its own, give what one after the other does."""
    out = []
    for together in (False, True):
        runs = [_make(2, 40, 64, seed=s) for s in (1, 2)]
        streams = [torch.cuda.Stream() for _ in runs]
        torch.cuda.synchronize()
        results = []
        for (block, tables, r), s in zip(runs, streams):
            with torch.cuda.stream(s):
                for new in ([20, 3], [1, 1], [1, 1]):
                    T = sum(new)
                    residual = r(T, block.hidden)
                    x, y = torch.empty(T, block.hidden, dtype=BF, device="cuda"), torch.empty(T, block.hidden, dtype=BF, device="cuda")
                    tables.step(torch.tensor(new, dtype=I32, device="cuda"))
                    block.pre(residual, x)
                    block.forward(residual, x, y, tables)
                    results.append(residual)
            if not together:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        out.append(results)
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_refusals(lib):
    block, tables, r = _make(2, 20, 64)
    x = torch.zeros(21, block.hidden, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        block.forward(x.float(), x, x.clone(), tables)
    small = moe.PageTables(block.cache, 2, 4, 4)
    with pytest.raises(ValueError):
        block.forward(x[:8].float(), x[:8], x[:8].clone(), small)
    with pytest.raises((TypeError, ValueError)):
        moe.AttentionBlock(block.cache, 8, 512, *block.weights, block.cos_sin, 2, 20, 4)


def test_example(lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "decoder.py"), "--hidden", "512", "--layers", "2",
                        "--requests", "2", "--prompt", "21", "--steps", "3"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "step 2" in r.stdout
