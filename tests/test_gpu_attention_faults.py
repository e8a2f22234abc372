"""Attention over the four-bit cache where single entries of its inputs are out of the ordinary: page ids that
are none, scales far apart, probabilities far apart, values that are NaN.  Against softmax in fp64, with a
bound for each row and channel that knows only what that row sees.

Tolerance.  Scores: as in test_gpu_attention.py, off by d <= 2^-19 sum |q k| scale, so a weight by
exp(2 d) - 1 <= 4 d of itself (d small); 2^-16 for exponentials and sums.  Probabilities are rounded to fp16,
2^-11 of themselves.  They are held as 2^(score - ref), a row's largest as 2^11 at least, or 2^6 with more than 32 rows
(2^7, ref is whole there).  Where they fall below 2^-14 they are off by half of fp16's smallest step, 2^-25, and of many
rows again wherever they are scaled down with ref, by 2 and more each time: 2^-25 / 2^11 = 2^-36 and 2 2^-25 / 2^6 = 2^-30 of
the row's largest: least.  So a row's channel is off by sum_j |v_j| (w_j (2^-11 + 4 d + 2^-16) + least max_i w_i), by
2^-24 of sum_j w_j |v_j| for the sum in fp32, and by half a step of the output's type; nothing that the row does not
see adds to it."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from _gpu_common import build_library
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _i(v):
    return torch.tensor(np.asarray(v), dtype=I32, device="cuda")


def _strict(case, out, lse=None, window=0, lost=(), only=None):
    """Every row and channel within the bound.  lost: (request, first token, end) that are not seen."""
    c, at = case, 0
    G, scale = c.Hq // c.Hk, c.D ** -0.5
    half = 2.0 ** -8 if out.dtype == BF else 2.0 ** -24
    for b, (L, n) in enumerate(zip(c.lens, c.news)):
        rows, at = slice(at, at + n), at + n
        if n == 0 or (only is not None and b not in only):
            continue
        k, v = c.values(b)
        q = c.q[rows].double().reshape(n, c.Hk, G, c.D)
        j, p = torch.arange(L, device="cuda"), torch.arange(L - n, L, device="cuda")[:, None]
        seen = (j[None] <= p) & ((j[None] > p - window) if window else True)
        for r, first, end in lost:
            if r == b:
                seen = seen & ~((j >= first) & (j < end))[None]
        seen = seen[:, None, None]
        x = torch.where(seen, torch.einsum("nhgd,hld->nhgl", q, k) * scale, -math.inf)
        d = torch.where(seen, torch.einsum("nhgd,hld->nhgl", q.abs(), k.abs()) * scale * 2.0 ** -19, 0.0)
        d = d.amax(-1, keepdim=True)
        z = torch.logsumexp(x, -1, keepdim=True)
        w = torch.exp(x - z)
        least = 2.0 ** (-30 if n * G > 32 else -36)
        off = w * (2.0 ** -11 + 4 * d + 2.0 ** -16 + 2.0 ** -24) + torch.where(seen, least * w.amax(-1, keepdim=True), 0.0)
        va = v.abs()
        ref, bound = torch.einsum("nhgl,hld->nhgd", w, v), torch.einsum("nhgl,hld->nhgd", off, va)
        got = out[rows].double().reshape(ref.shape)
        err, bound = (got - ref).abs(), bound + ref.abs() * half
        assert bool((err <= bound).all()), (b, float((err / bound.clamp(min=1e-300)).max()))
        if lse is not None:
            zz, gz = z[..., 0], lse[rows].double().reshape(z.shape[:-1])
            assert bool(((gz - zz).abs() <= d[..., 0] + 2.0 ** -20 * (1 + zz.abs())).all())


def _forward(case, dtype=F32, status=0, window=0, table=None):
    out = torch.full(case.q.shape, 7.0, dtype=dtype, device="cuda")
    lse = torch.full(case.q.shape[:2], 7.0, device="cuda")
    word = _i([0])
    case.plan(window=window).forward(case.q, case.table if table is None else table, case.lengths, case.starts, out,
                                     lse=lse, status=word)
    assert int(word) == status
    return out, lse


@pytest.mark.parametrize("news", [[2, 1], [40, 3], [3, 300]])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 64)])
@pytest.mark.parametrize("bad", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1, "pages"])
def test_page_ids_that_are_none(lib, news, D, page, bad):
    """Their tokens are not seen, whatever the id is, and the status says so."""
    lens = [n + 150 for n in news]
    c = Case(lens, news, 8, 2, D, page, seed=2)
    table = c.table.clone()
    table[0, 1] = table[1, 0] = c.cache.pages if bad == "pages" else bad
    out, lse = _forward(c, status=moe.DEV_BAD_INDEX, table=table)
    _strict(c, out, lse, lost=[(0, page, 2 * page), (1, 0, page)])


ROWS = [[3], [40], [300]]   # query tokens of a request: 12 rows of a head, many rows, rows of several groups


@pytest.mark.parametrize("news", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("more", [27, 40, 100])
@pytest.mark.parametrize("where", [0, 130, -2])
def test_one_key_far_above_the_others(lib, news, D, more, where):
    """A block of one key 2^more above the others: scores of the other keys are what they were, for rows that see
    it and rows that stand before it."""
    c = Case([news[0] + 200], news, 8, 2, D, 16, seed=more)
    at = where % c.lens[0]
    p, o = int(c.host_table[0, at // 16]), at % 16
    c.cache.scales[p, 0, :, o, 1] += more
    if where >= 0:
        c.q[..., 32:64] = 0   # all rows see it; it gives scores of nothing
    out, lse = _forward(c)
    if where >= 0:
        _strict(c, out, lse)
    else:   # the last two rows' scores have no meaning beside 2^100; all rows before are as they were
        c.lens, c.news = [at], [news[0] - 2]
        _strict(c, out, lse)


@pytest.mark.parametrize("news", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shift", [-100, -30, 14, 16, 18, 60, 100])
def test_keys_of_any_size(lib, news, D, shift):
    """Keys times 2^shift and queries times 2^-shift: the same scores."""
    c = Case([news[0] + 77], news, 8, 2, D, 32, seed=shift + 100)
    c.poison_stale()
    scales = c.cache.scales[:, 0]
    c.cache.scales[:, 0] = torch.where(scales == 255, 255, scales.int() + shift).to(torch.uint8)
    c.q *= 2.0 ** -shift
    _strict(c, *_forward(c))


@pytest.mark.parametrize("news", [[3], [60, 1], [300]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("light", [False, True])
def test_a_value_that_is_nan(lib, news, D, window, light):
    """Reaches the rows that see it, in its block of channels, also where its weight is next to nothing (2^-43 and
    less); keys and queries that are NaN reach all of a row.  The others keep their bits."""
    lens = [n + 250 for n in news]
    c = Case(lens, news, 8, 2, D, 16, seed=3)
    n, L, at = news[0], lens[0], lens[0] - 2 if news[0] < 60 else lens[0] - 50
    p, o = int(c.host_table[0, at // 16]), at % 16
    if light:   # every row's score there is 30 below zero, others' near it
        c.q[..., :32] = 3.75 * D ** 0.5
        c.q[..., 32:] *= 0.1
        c.cache.scales[:, 0, :, :, 0] = 110
        c.cache.codes[p, 0, :, o, :16] = 0x99   # -0.5 each
        c.cache.scales[p, 0, :, o, 0] = 126
    kw = dict(window=window)
    clean, _ = _forward(c, **kw)
    pos = torch.arange(L - n, L, device="cuda")
    sees = (pos >= at) & ((pos - window < at) if window else True)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    c.cache.scales[p, 1, 1, o, D // 32 - 1] = 255
    c.cache.codes[p, 1, 1, o, D // 2 - 16:] = 0
    bad[:n, 4:, D - 32:] = sees[:, None, None]
    out, _ = _forward(c, **kw)
    assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == clean[~bad]).all())
    c.cache.scales[p, 0, 0, o, 1] = 255
    c.cache.codes[p, 0, 0, o, 16:32] = 0
    bad[:n, :4] |= sees[:, None, None]
    out, _ = _forward(c, **kw)
    assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == clean[~bad]).all())
    c.q[n - 1, 2, 5] = float("nan")
    bad[n - 1, 2] = True
    out, _ = _forward(c, **kw)
    assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == clean[~bad]).all())


def test_a_value_that_is_nan_in_requests_cut_between_ctas(lib):
    for news in ([1], [40]):
        c = Case([20001], news, 8, 1, 128, 64, seed=7)
        clean, _ = _forward(c)
        p, o = int(c.host_table[0, 9000 // 64]), 9000 % 64
        c.cache.scales[p, 1, 0, o, 2], c.cache.codes[p, 1, 0, o, 32:48] = 255, 0
        out, _ = _forward(c)
        assert bool(torch.isnan(out[..., 64:96]).all())
        assert bool((out[..., :64] == clean[..., :64]).all()) and bool((out[..., 96:] == clean[..., 96:]).all())


@pytest.mark.parametrize("news", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("more", [20, 30, 90])
@pytest.mark.parametrize("where", [0, 130, -2])
def test_one_value_far_above_the_others(lib, news, D, more, where):
    """A block of one value 2^more above the others: rows that stand before it and other channels are as they were."""
    c = Case([news[0] + 200], news, 8, 2, D, 16, seed=more)
    c.poison_stale()
    at = where % c.lens[0]
    p, o = int(c.host_table[0, at // 16]), at % 16
    c.cache.scales[p, 1, :, o, 1] += more
    _strict(c, *_forward(c))


@pytest.mark.parametrize("news", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shift", [-110, -40, -28, 8, 12, 30, 90])
def test_values_of_any_size(lib, news, D, shift):
    """All values times 2^shift, with a token whose values are zero (its blocks' scale is 1) among them."""
    c = Case([news[0] + 77], news, 8, 2, D, 32, seed=shift + 110)
    c.poison_stale()
    scales = c.cache.scales[:, 1]
    c.cache.scales[:, 1] = torch.where(scales == 255, 255, scales.int() + shift).to(torch.uint8)
    p = int(c.host_table[0, 1])
    c.cache.scales[p, 1, :, 5], c.cache.codes[p, 1, :, 5] = 127, 0
    _strict(c, *_forward(c))


@pytest.mark.parametrize("news", [[3], [40], [300], [1, 70, 4]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("share", [0.002, 0.05, 1.0])
@pytest.mark.parametrize("window", [0, 150])
def test_values_of_all_sizes_together(lib, news, D, share, window):
    """Scale bytes of 2 to 220 for a share of the blocks: every row and channel to what its own terms allow."""
    c = Case([n + 500 for n in news], news, 8, 2, D, 16, seed=D)
    c.poison_stale()
    g = torch.Generator(device="cuda").manual_seed(1)
    s = c.cache.scales[:, 1]
    odd = (torch.rand(s.shape, device="cuda", generator=g) < share) & (s != 255)
    c.cache.scales[:, 1] = torch.where(odd, torch.randint(2, 221, s.shape, device="cuda", generator=g).to(torch.uint8), s)
    _strict(c, *_forward(c, window=window), window=window)


def test_values_of_all_sizes_in_requests_cut_between_ctas(lib):
    for news, D in (([1], 128), ([5], 64), ([40], 128)):
        c = Case([30001], news, 8, 1, D, 64, seed=7)
        g = torch.Generator(device="cuda").manual_seed(2)
        s = c.cache.scales[:, 1]
        odd = torch.rand(s.shape, device="cuda", generator=g) < 0.001
        c.cache.scales[:, 1] = torch.where(odd, torch.randint(60, 180, s.shape, device="cuda", generator=g).to(torch.uint8), s)
        _strict(c, *_forward(c))


@pytest.mark.parametrize("news", ROWS + [[1, 50]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("below", [8, 12, 15, 18])
@pytest.mark.parametrize("where", [0, 8000])
def test_results_of_probabilities_far_below_the_largest(lib, news, D, below, where):
    """One key `below` natural logarithms above 8000 others, and its values zero: the others are the result."""
    c = Case([8100 + n for n in news], news, 8, 2, D, 64, seed=below)
    c.cache.scales[:, 0, :, :, 0] = 127
    c.cache.codes[:, 0, :, :, :16] = 0xbb   # -1.5 each
    c.q[..., :32] = below * D ** 0.5 / 96
    c.q[..., 32:] *= 0.3
    c.cache.codes[:, 1] &= 0x77   # no value below zero: nothing cancels
    for b in range(len(news)):
        p, o = int(c.host_table[b, where // 64]), where % 64
        c.cache.codes[p, 0, :, o, :16] = 0x33   # 1.5
        c.cache.codes[p, 1, :, o] = 0
    _strict(c, *_forward(c))


@pytest.mark.parametrize("news", ROWS)
@pytest.mark.parametrize("step", [1, 3, 13, 40])
def test_scores_that_rise_all_the_way(lib, news, step):
    """Scores that grow by `step` (log2) every 32 or 16 tokens, so that the maximum rises within and between tiles."""
    c = Case([900], news, 8, 2, 128, 16, seed=step)
    c.cache.scales[:, 0, :, :, 0] = 127
    c.cache.codes[:, 0, :, :, :16] = 0
    tokens = np.arange(900)
    page, off = c.host_table[0, tokens // 16], tokens % 16
    # a channel of the first block for each bit of the count of 16 tokens: 1 or 0 there, 2^bit in q
    codes = np.zeros((900, 16), np.uint8)
    for bit in range(6):
        codes[:, bit] = np.where((tokens // 16) >> bit & 1, 0x02, 0)
    c.cache.codes[torch.tensor(page), 0, :, torch.tensor(off), :16] = torch.tensor(codes, device="cuda")[:, None]
    c.q *= 0.1
    c.q[..., :32] = 0
    for bit in range(6):
        c.q[..., 2 * bit] = step * 2.0 ** bit * 128 ** 0.5 * 0.6931
    _strict(c, *_forward(c))
