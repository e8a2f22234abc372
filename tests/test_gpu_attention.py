"""Attention over the four-bit cache against softmax in fp64, over what the cache holds.

Tolerance.  Scores: products of bf16 queries and cached keys are exact, sums fp32 in the tensor cores
(16 terms at a time, truncated: 2^-23 each) and over four blocks: off by d <= 2^-19 sum |q k| scale.
Probabilities carry that, the hardware's exponential (2^-22) and their rounding to fp16 (2^-11).  So the
output is off by at most A (2^-11 + 4 d + 2^-16), A the mean of |v| with the row's weights, by 2^-20 of the
largest |v| (values whose block scale is 2^-22 of it count as zero, and probabilities below 2^-24 lose
bits), and by half a step of its type (2^-8 for bf16)."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from oracle import mx4

from _gpu_common import build_library

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _i(v):
    return torch.tensor(np.asarray(v), dtype=I32, device="cuda")


class Case:
    """A filled cache with pages anywhere, stale rows behind each request's last token."""

    def __init__(self, lens, news, Hq, Hk, D, page, seed=0, kscale=1.0, extra_rows=0, columns=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        order = r.permutation(pages)
        table = np.full((len(lens), max(need + [0]) + columns), -1)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.kv = torch.randn(pages, 2, Hk, page, D, device="cuda", generator=g)
        self.kv *= torch.exp(0.5 * torch.randn(pages, 2, Hk, page, 1, device="cuda", generator=g))
        self.kv[:, 0] *= kscale
        codes, scales = moe.mx4_quantize(self.kv.bfloat16())
        self.cache = moe.Cache4.of(codes, scales)
        self.lens, self.news, self.Hq, self.Hk, self.D, self.page = lens, news, Hq, Hk, D, page
        self.host_table = table
        rows = sum(news) + extra_rows
        self.q = torch.randn(rows, Hq, D, device="cuda", generator=g).bfloat16()
        self.table, self.lengths, self.starts = _i(table), _i(lens), _i(np.concatenate([[0], np.cumsum(news)]))

    def poison_stale(self):
        """What lies behind the last tokens becomes NaN (the cache's rows that nothing was written to)."""
        for b, L in enumerate(self.lens):
            if L % self.page:
                p = int(self.host_table[b, L // self.page])
                self.cache.scales[p, :, :, L % self.page:] = 255
                self.cache.codes[p, :, :, L % self.page:] = 0x77

    def plan(self, **kw):
        return moe.CacheAttention(len(self.lens), self.q.shape[0], self.Hq, self.cache, self.table.shape[1],
                                  max_q=max(self.news + [1]), max_len=max(self.lens + [1]), **kw)

    def values(self, b):
        """keys, values fp64 [Hk, len, D] of request b."""
        L = self.lens[b]
        if L == 0:
            return torch.zeros(2, self.Hk, 0, self.D, dtype=torch.float64, device="cuda")
        pos = np.arange(L)
        ids = torch.tensor(self.host_table[b, pos // self.page], device="cuda")
        off = torch.tensor(pos % self.page, device="cuda")
        c, s = self.cache.codes[ids, :, :, off].cpu().numpy(), self.cache.scales[ids, :, :, off].cpu().numpy()
        v = torch.tensor(mx4.dequantize(c, s), device="cuda")   # [L, 2, Hk, D]
        return v[:, 0].transpose(0, 1), v[:, 1].transpose(0, 1)

    def check(self, out, lse=None, window=0, scale=None, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        G, at = self.Hq // self.Hk, 0
        half = 2.0 ** -8 if out.dtype == BF else 2.0 ** -24
        for b, (L, n) in enumerate(zip(self.lens, self.news)):
            rows, at = slice(at, at + n), at + n
            if n == 0 or (only is not None and b not in only):
                continue
            k, v = self.values(b)
            q = self.q[rows].double().reshape(n, self.Hk, G, self.D)
            x = torch.einsum("nhgd,hld->nhgl", q, k) * scale
            d = 2.0 ** -19 * scale * torch.einsum("nhgd,hld->nhgl", q.abs(), k.abs())
            p = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None]
            seen = (j <= p) & ((j > p - window) if window else True)
            x = torch.where(seen[:, None, None], x, -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            w = torch.where(torch.isfinite(z), torch.exp(x - z), 0.0)
            ref = torch.einsum("nhgl,hld->nhgd", w, v)
            mean = torch.einsum("nhgl,hld->nhgd", w, v.abs())
            dmax = torch.where(seen[:, None, None], d, 0.0).amax(-1, keepdim=True) if L else torch.zeros_like(z)
            vmax = v.abs().amax() if L else 0.0
            bound = mean * (2.0 ** -11 + 4 * dmax + 2.0 ** -16) + vmax * 2.0 ** -20 + ref.abs() * half
            got = out[rows].double().reshape(ref.shape)
            err = (got - ref).abs()
            assert bool((err <= bound).all()), (b, float((err / bound.clamp(min=1e-300)).max()))
            if lse is not None:
                zz, gz = z[..., 0], lse[rows].double().reshape(z.shape[:-1])
                assert bool((torch.isinf(zz) == torch.isinf(gz)).all())
                fin = torch.isfinite(zz)
                assert bool(((gz - zz).abs()[fin] <= (dmax[..., 0] + 2.0 ** -20 * (1 + zz.abs()))[fin]).all())


def _run(case, out_dtype=BF, lse=False, window=0, scale=None):
    out = torch.full(case.q.shape, 7.0, dtype=out_dtype, device="cuda")
    z = torch.full(case.q.shape[:2], 7.0, device="cuda") if lse else None
    status = _i([0])
    case.plan(window=window, scale=scale).forward(case.q, case.table, case.lengths, case.starts, out, lse=z, status=status)
    assert int(status) == 0
    case.check(out, z, window, scale)
    return out, z


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 127, 128, 129, 500, 3001])
@pytest.mark.parametrize("D", [64, 128])
def test_one_token_of_one_request(lib, L, D):
    c = Case([L], [1], 8, 1, D, 16, seed=L)
    c.poison_stale()
    _run(c, lse=True)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (5, 1), (7, 7), (16, 2), (12, 4), (24, 1), (40, 8), (64, 2), (64, 1)])
@pytest.mark.parametrize("D,page", [(64, 32), (128, 128)])
def test_head_layouts(lib, Hq, Hk, D, page):
    c = Case([70, 333], [1, 1], Hq, Hk, D, page, seed=Hq)
    c.poison_stale()
    _run(c, out_dtype=F32, lse=True)


@pytest.mark.parametrize("news", [[2], [3, 1, 5], [9, 4], [1, 33, 2], [100], [257, 1, 64]])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (5, 1, 64), (4, 4, 128)])
def test_several_query_tokens(lib, news, Hq, Hk, D):
    lens = [n + 41 * i + (0 if i % 2 else 60) for i, n in enumerate(news)]
    c = Case(lens, news, Hq, Hk, D, 16, seed=sum(news))
    c.poison_stale()
    _run(c, lse=True)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000])
@pytest.mark.parametrize("news", [[1, 1], [4, 60]])
def test_windows(lib, window, news):
    c = Case([300, 611], news, 6, 2, 128, 32, seed=window)
    _run(c, lse=True, window=window)


def test_a_batch_of_every_length(lib):
    lens = list(range(1, 60)) + [1000, 5000, 64, 4096]
    c = Case(lens, [1] * len(lens), 16, 2, 128, 64)
    c.poison_stale()
    _run(c)


def test_long_requests_cut_between_many_ctas(lib):
    c = Case([40001, 3, 25000], [1, 1, 2], 8, 1, 128, 16, seed=3)
    _run(c, lse=True)
    c = Case([70000], [1], 4, 4, 64, 128, seed=4)
    _run(c)


def test_rows_that_see_nothing_empty_requests_and_rows_behind(lib):
    """Positions below zero, requests without query tokens, rows that belong to no request."""
    c = Case([5, 0, 20, 0, 1], [2, 0, 0, 3, 1], 4, 2, 128, 16, extra_rows=3)
    c.lens[0] = 1   # two query tokens and one cached: the first sees nothing
    c.lengths[0] = 1
    out, z = _run(c, lse=True)
    assert not bool(out[0].any()) and bool(torch.isinf(z[0]).all()) and bool((z[0] < 0).all())
    assert not bool(out[2:5].any()) and bool(torch.isinf(z[2:5]).all())
    assert bool((out[6:] == 7).all()) and bool((z[6:] == 7).all())


@pytest.mark.parametrize("news", [[1, 1, 1], [5, 40, 1]])
def test_bad_requests_and_pages(lib, news):
    """A request that cannot be right is not computed; tokens of a page that is not there are not seen."""
    lens = [100, 200, 90]
    c = Case(lens, news, 8, 2, 128, 16)
    plan, out = c.plan(), torch.full(c.q.shape, 7.0, dtype=BF, device="cuda")
    status = _i([0])
    lengths = c.lengths.clone()
    lengths[0], lengths[2] = -1, c.table.shape[1] * 16 + 1
    plan.forward(c.q, c.table, lengths, c.starts, out, status=status)
    assert int(status) == moe.DEV_BAD_INDEX
    c.check(out, only=[1])
    a, b = c.starts.tolist()[1:3]
    assert bool((out[:a] == 7).all()) and bool((out[b:] == 7).all())
    status.zero_()
    starts = c.starts.clone()
    starts[3] = c.q.shape[0] + 1
    out.fill_(7.0)
    plan.forward(c.q, c.table, c.lengths, starts, out, status=status)
    assert int(status) == moe.DEV_BAD_INDEX
    c.check(out, only=[0, 1])
    # pages: the last tokens' first page is nowhere; without its tokens the rest is as if they were masked
    for bad in (-1, c.cache.pages, 1 << 30):
        status.zero_()
        table = c.table.clone()
        table[1, 2] = bad
        got = plan.forward(c.q, table, c.lengths, c.starts, torch.empty_like(out), status=status)
        assert int(status) == moe.DEV_BAD_INDEX
        c.check(got, only=[0, 2])
        lost = Case(lens, news, 8, 2, 128, 16)   # the same, with scores of minus infinity there
        k, v = lost.values(1)
        G, n = 4, news[1]
        q = lost.q[a:b].double().reshape(n, 2, G, 128)
        x = torch.einsum("nhgd,hld->nhgl", q, k) * 128 ** -0.5
        j = torch.arange(200, device="cuda")
        hidden = (j[None] > torch.arange(200 - n, 200, device="cuda")[:, None]) | ((j >= 32) & (j < 48))[None]
        w = torch.softmax(x.masked_fill(hidden[:, None, None], -math.inf), -1)
        ref = torch.einsum("nhgl,hld->nhgd", w, v).reshape(n, 8, 128)
        assert float((got[a:b].double() - ref).abs().max()) < 2e-2 * float(ref.abs().max())


def test_large_and_small_scores(lib):
    c = Case([900], [3], 8, 2, 128, 16, kscale=30.0)   # a softmax of nearly one token
    _run(c, lse=True)
    c = Case([900], [3], 8, 2, 128, 16, kscale=1e-6)   # all tokens alike
    _run(c, lse=True)
    c = Case([900], [1], 8, 2, 64, 16, seed=9)
    c.q *= 1e4
    _run(c, scale=1e-5)
    c.q *= 0
    _run(c, lse=True)


@pytest.mark.parametrize("news", [[2], [60]])
def test_scores_far_below_and_above_zero(lib, news):
    """All scores of a row at -1000 or 1000: what stands before its first token must not matter."""
    for sign in (-1.0, 1.0):
        c = Case([500], news, 8, 2, 128, 16, seed=13)
        c.cache.codes[:, 0, :, :, :16] = 0x33   # 1.5 each
        c.cache.codes[:, 0, :, :, 16:] &= 0x11
        c.cache.scales[:, 0] = 127
        c.q[..., :32] = sign * 20.0 * c.D ** 0.5
        c.q[..., 32:] *= 0.1
        _run(c, lse=True)
        _run(c, lse=True, window=100)


def test_values_of_very_different_sizes(lib):
    """A value 2^15 times the others', wherever it stands: the others still count."""
    for where in (0, 70, 799):
        c = Case([800], [2], 8, 1, 128, 16, seed=where)
        p, o = int(c.host_table[0, where // 16]), where % 16
        c.cache.scales[p, 1, 0, o, 1] += 15
        _run(c, out_dtype=F32)
        c.cache.scales[p, 1, 0, o, 1] += 40   # and one beside which they are nothing
        _run(c, out_dtype=F32)


def test_nan_and_infinity_reach_only_those_who_see_them(lib):
    c = Case([200, 200], [4, 1], 8, 2, 128, 16, seed=11)
    clean, _ = _run(c)
    # token 198 of request 0: rows 0 and 1 stand before it
    p = int(c.host_table[0, 198 // 16])
    c.cache.scales[p, 1, 1, 198 % 16, 2] = 255
    c.cache.codes[p, 1, 1, 198 % 16, 32:48] = 0
    plan = c.plan()
    out = plan.forward(c.q, c.table, c.lengths, c.starts, torch.empty_like(clean))
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[2:4, 4:, 64:96] = True
    assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == clean[~bad]).all())
    # a key: all channels of those heads
    c.cache.scales[p, 0, 0, 198 % 16, 2] = 255
    c.cache.codes[p, 0, 0, 198 % 16, 32:48] = 0
    out = plan.forward(c.q, c.table, c.lengths, c.starts, torch.empty_like(clean))
    bad[2:4, :4] = True
    assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == clean[~bad]).all())
    # a query
    c.q[4, 3, 7] = float("nan")
    out = plan.forward(c.q, c.table, c.lengths, c.starts, torch.empty_like(clean))
    bad[4, 3] = True
    assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == clean[~bad]).all())
    # outside a window: nothing of it
    c = Case([300], [1], 8, 2, 128, 16, seed=12)
    clean, _ = _run(c, window=50)
    p = int(c.host_table[0, 240 // 16])
    c.cache.scales[p, :, :, 0:10] = 255   # tokens 240 .. 249
    assert torch.equal(c.plan(window=50).forward(c.q, c.table, c.lengths, c.starts, torch.empty_like(clean)), clean)


@pytest.mark.parametrize("news", [[1, 1, 1], [70, 1, 20]])
def test_in_place_same_bits_graph_and_streams(lib, news):
    c = Case([700, 90, 2500], news, 16, 2, 128, 32, seed=5)
    want, _ = _run(c)
    plan, plan2 = c.plan(), c.plan()
    q = c.q.clone()
    assert plan.forward(q, c.table, c.lengths, c.starts, q) is q and torch.equal(q, want)
    out, out2 = torch.empty_like(want), torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):   # two streams at once, each with its own workspace
        plan.forward(c.q, c.table, c.lengths, c.starts, out)
        plan2.forward(c.q, c.table, c.lengths, c.starts, out2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(out2, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.forward(c.q, c.table, c.lengths, c.starts, out)
    # lengths change between replays
    short = Case([650, 80, 2400], news, 16, 2, 128, 32, seed=5)
    c.lengths.copy_(short.lengths)
    g.replay()
    c.lens = short.lens
    c.check(out)


def test_more_rows_on_the_device_than_the_plan_was_made_for(lib):
    c = Case([300, 900], [40, 70], 8, 1, 128, 16, seed=6)
    plan = moe.CacheAttention(2, 110, 8, c.cache, c.table.shape[1], max_q=1, max_len=16)
    out = plan.forward(c.q, c.table, c.lengths, c.starts, torch.empty_like(c.q))
    c.check(out)


def test_no_requests_and_no_rows(lib):
    c = Case([16], [1], 4, 1, 64, 16)
    z = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    moe.CacheAttention(1, 0, 4, c.cache, 2).forward(z, _i([[0, 0]]), _i([16]), _i([0, 0]), z)
    moe.CacheAttention(0, 0, 4, c.cache, 2).forward(z, _i(np.zeros((0, 2))), _i([]), _i([0]), z)
