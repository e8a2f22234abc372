"""Calls at the edges of what attention's operators take: page ids whose slots are no numbers, windows
longer than any request, tensors of another device, one workspace for calls of many sizes, products
that many clusters share.  (Tolerances: test_gpu_attention.py, test_gpu_w4.py.)"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from moe_expert_layer_07_gb300 import attention as A

from _gpu_common import build_library
from test_gpu_attention import Case
from test_gpu_cache import _call, _i
from test_gpu_decoder import _make

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "first"])
def test_free_pages_that_are_none(lib, page, bad):
    """Their tokens' slots are in no cache: not those of another page, and not -1, which is taken for padding."""
    if bad == "first":
        bad = (2 ** 31 - 1) // page + 1   # its slots would be those of page 0
    got = _call([0, 3], [3, 2], np.array([[-7, -7], [5, -7]]), [bad, 9], 0, 2, page, 7)
    assert list(got["slots"]) == [-2 ** 31] * 3 + [5 * page + 3, 5 * page + 4, -1, -1]
    assert got["table"][0, 0] == bad and list(got["lengths"]) == [3, 5]
    cache = moe.Cache4(12, page, 1, 64)
    cache.codes.fill_(1), cache.scales.fill_(7)
    status = _i([0])
    qkv = torch.randn(7, 3 * 64, device="cuda").bfloat16()
    q = torch.zeros(7, 1, 64, dtype=BF, device="cuda")
    moe.qk_norm_rope(qkv, None, None, 1, 1, q, cache=cache, slots=_i(got["slots"]), status=status)
    assert int(status) == moe.DEV_BAD_INDEX
    assert bool((cache.scales[:5] == 7).all()) and bool((cache.codes[6:] == 1).all())


@pytest.mark.parametrize("in_place", [False, True])
def test_a_held_page_that_is_none(lib, in_place):
    table = np.array([[2 ** 31 // 16, -7]])
    status = _i([0])
    got = _call([3], [2], table, [4], 0, 1, 16, 3, status, in_place)
    assert int(status) == moe.DEV_BAD_INDEX and list(got["lengths"]) == [3] and list(got["slots"]) == [-1] * 3


@pytest.mark.parametrize("window", [48, 96, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("news", [[3, 1], [60, 7]])
def test_windows_longer_than_the_requests(lib, window, news):
    """The same bits as without one, rows before the first token among them."""
    case = Case([40, 5], news, 8, 1, 128, 16)
    outs = []
    for w in (0, window):
        out = torch.full_like(case.q, 3.0)
        case.plan(window=w).forward(case.q, case.table, case.lengths, case.starts, out)
        outs.append(out)
    case.check(outs[0])
    assert torch.equal(*outs)


def test_fewer_rows_in_the_same_workspace(lib):
    case = Case([300, 77], [90, 30], 8, 2, 64, 32)
    big = moe.CacheAttention(2, 400, 8, case.cache, case.table.shape[1], max_q=90, max_len=300)
    plan = big.of_rows(120)
    assert plan.ws is big.ws and big.d.rows == 400
    out = torch.empty_like(case.q)
    plan.forward(case.q, case.table, case.lengths, case.starts, out)
    case.check(out)
    for rows in (-1, 401):
        with pytest.raises(ValueError):
            big.of_rows(rows)


def test_a_block_keeps_one_workspace(lib):
    block, tables, r = _make(2, 48, 512)
    x = torch.zeros(48, block.hidden, dtype=BF, device="cuda")
    residual, y = x.float(), torch.empty_like(x)
    before = None
    for T in range(1, 49):
        tables.step(_i([1, 1] if T > 1 else [1, 0]))
        block.forward(residual[:T], x[:T], y[:T], tables)
        if T == 20:
            torch.cuda.synchronize()
            before = torch.cuda.memory_allocated()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before < 1 << 20
    assert all(p.ws is block.plan.ws for p in block._plans.values())
    assert int(tables.status) == 0 and block.status() == 0


def test_a_block_on_a_stream_given_as_an_address(lib):
    outs = []
    for raw in (False, True):
        block, tables, r = _make(1, 40, 64)
        s = torch.cuda.Stream()
        residual, x, y = r(20, block.hidden), r(20, block.hidden).bfloat16(), torch.empty(20, block.hidden, dtype=BF, device="cuda")
        new = _i([20])
        torch.cuda.synchronize()
        stream = s.cuda_stream if raw else s
        tables.step(new, stream)
        block.forward(residual, x, y, tables, stream=stream)
        torch.cuda.synchronize()
        outs.append(residual)
    assert torch.equal(*outs)


def test_tensors_of_another_device_are_refused(lib, monkeypatch):
    """As seen from device 1: nothing of the calls is launched."""
    case = Case([20], [2], 4, 2, 64, 16)
    plan = case.plan()
    out, slots = torch.full_like(case.q, 3.0), _i([0, 1])
    x, w = torch.ones(2, 64, dtype=BF, device="cuda"), torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s, y = torch.full((8, 2), 127, dtype=torch.uint8, device="cuda"), torch.full((2, 8), 3.0, device="cuda")
    qkv, k = torch.ones(2, 8 * 64, dtype=BF, device="cuda"), torch.full((2, 2, 64), 3.0, dtype=BF, device="cuda")
    tables = moe.PageTables(case.cache, 2, 3, 4)
    calls = [lambda: plan.forward(case.q, case.table, case.lengths, case.starts, out),
             lambda: moe.w4_matvec(x, w, s, y), lambda: moe.cache_read(case.cache, slots, k, None),
             lambda: moe.qk_norm_rope(qkv, None, None, 4, 2, out, k_out=k),
             lambda: tables.step(_i([1, 1]))]
    monkeypatch.setattr(A, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="device"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert all(bool((t == 3.0).all()) for t in (out, y, k)) and not tables.lengths.any()
    for call in calls:
        call()


@pytest.mark.parametrize("T,N,K", [(1, 4100, 16384), (16, 1000, 24576), (3, 5003, 32768), (9, 2500, 20480)])
def test_products_of_clusters_of_every_size(lib, T, N, K):
    """More row tiles than clusters that run at once, several exchanges of sums to a cluster."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    codes, scales = moe.mx4_quantize(torch.randn(N, K, device="cuda", generator=g).bfloat16())
    out = torch.empty(T, N, device="cuda")
    moe.w4_matvec(x, codes, scales, out)
    w = moe.mx4_dequantize(codes, scales).double()
    ref, size = x.double() @ w.t(), x.double().abs() @ w.t().abs()
    bound = 2.0 ** -17 * size + 2.0 ** -24 * ref.abs() + 2.0 ** -29 * x.double().abs().amax(1, keepdim=True) * w.abs().sum(1)
    assert bool(((out.double() - ref).abs() <= bound).all())
    again = torch.empty_like(out)
    moe.w4_matvec(x, codes, scales, again)
    assert torch.equal(out, again)


def test_calls_of_several_threads(lib):
    """Sizes that ask for different amounts of shared memory, launched at the same time."""
    import threading
    cases = [Case([40] * n, [1] * n, 8, 1, 128, 16, seed=n) for n in (1, 700)]
    x = torch.randn(2, 8192, device="cuda").bfloat16()
    failed, outs = [], {}

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                case, plan = cases[i], cases[i].plan()
                codes = torch.full((64, (4096 >> i) // 2), 0x21, dtype=torch.uint8, device="cuda")
                scales = torch.full((64, (4096 >> i) // 32), 127, dtype=torch.uint8, device="cuda")
                out, y = torch.empty_like(case.q), torch.empty(2, 64, device="cuda")
                xi = x[:, :4096 >> i].contiguous()
                for _ in range(300):
                    plan.forward(case.q, case.table, case.lengths, case.starts, out)
                    moe.w4_matvec(xi, codes, scales, y)
                torch.cuda.current_stream().synchronize()
                outs[i] = out
        except Exception as e:   # noqa: BLE001
            failed.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for i, case in enumerate(cases):
        case.check(outs[i])


def _mx4_64(v):
    """MXFP4 of fp64 values [..., D]: codes [..., D], scale bytes [..., D/32] (no ties among random values)."""
    b = v.reshape(v.shape[:-1] + (-1, 32))
    most = b.abs().amax(-1)
    byte = torch.where(most > 0, (torch.frexp(most).exponent - 1 - 2 + 127).clamp(min=0), 127)
    y = b.abs() * torch.exp2(127.0 - byte.double()).unsqueeze(-1)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=v.device)
    codes = torch.searchsorted(mid, y.contiguous()) + 8 * (b < 0)
    return codes.reshape(v.shape), byte


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("D,R,norm", [(128, 128, True), (64, 32, True), (64, 64, False), (128, 0, True)])
def test_cached_keys_are_the_codes_of_exact_values(lib, style, D, R, norm):
    """Not those of values that rounding put on the other side of a border between codes, or of a power of two."""
    T, Hk = 30000 * 128 // D, 8
    g = torch.Generator(device="cuda").manual_seed(D + R + style)
    qkv = torch.randn(T, 3 * Hk * D, device="cuda", generator=g).bfloat16()
    w = (1 + 0.1 * torch.randn(D, device="cuda", generator=g)).bfloat16() if norm else None
    pos = torch.randint(1, 8000, (T,), device="cuda", generator=g).to(I32)
    cs = moe.rope_table(8000, R) if R else None
    cache = moe.Cache4(-(-T // 64), 64, Hk, D)
    q = torch.empty(T, Hk, D, dtype=BF, device="cuda")
    moe.qk_norm_rope(qkv, pos, cs, Hk, Hk, q, w_k=w, cache=cache, slots=torch.arange(T, device="cuda", dtype=I32), style=style)
    at = torch.arange(T, device="cuda")
    for h in range(Hk):
        v = qkv[:, (Hk + h) * D:(Hk + h + 1) * D].double()
        if norm:
            v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w.double()
        if R:
            c, s = cs.double()[pos.long()][:, :R // 2], cs.double()[pos.long()][:, R // 2:]
            if style == 0:
                a, b = v[:, :R // 2], v[:, R // 2:R]
                v = torch.cat([a * c - b * s, b * c + a * s, v[:, R:]], -1)
            else:
                a, b = v[:, 0:R:2], v[:, 1:R:2]
                v = torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(1), v[:, R:]], -1)
        codes, byte = _mx4_64(v)
        got, scale = cache.codes[at // 64, 0, h, at % 64].long(), cache.scales[at // 64, 0, h, at % 64].long()
        got = torch.stack([got & 15, got >> 4], -1).flatten(1)
        assert torch.equal(scale, byte.long())
        if norm:   # (elsewhere exact ties are possible)
            assert torch.equal(got, codes)
        else:
            assert int((got != codes).sum()) <= 2


@pytest.mark.parametrize("new", [1, 2, 4, 5, 40])
@pytest.mark.parametrize("D,Hk", [(128, 2), (64, 1)])
def test_one_request_in_buffers_for_many_rows(lib, new, D, Hk):
    """What a plan of many rows does with few, and the calls of fewer rows in its workspace."""
    case = Case([333], [new], 8, Hk, D, 32, extra_rows=64 - new)
    big = moe.CacheAttention(1, 64, 8, case.cache, case.table.shape[1], max_q=64, max_len=400)
    for rows in sorted({64, new, 17}):
        if rows < new:
            continue
        out = torch.full_like(case.q[:rows], 3.0)
        lse = torch.full((rows, 8), 3.0, device="cuda")
        big.of_rows(rows).forward(case.q[:rows], case.table, case.lengths, case.starts, out, lse=lse)
        case.check(out, lse)
        assert bool((out[new:] == 3.0).all()) and bool((lse[new:] == 3.0).all())


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (9, 1), (40, 2), (48, 1)])
def test_a_workspace_holds_every_smaller_call(lib, Hq, Hk):
    """Head layouts whose calls of 1, 2, 3 .. rows take different kernels."""
    case = Case([70], [1], Hq, Hk, 64, 16, extra_rows=36)
    for most in (1, 2, 3, 5, 37):
        big = moe.CacheAttention(1, most, Hq, case.cache, case.table.shape[1], max_q=most, max_len=100)
        for rows in range(1, most + 1, 2):
            out = torch.empty_like(case.q[:rows])
            big.of_rows(rows).forward(case.q[:rows], case.table, case.lengths, case.starts, out)
            case.check(out)
