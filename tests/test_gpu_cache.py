"""The tables of the paged cache, the norm and rotation before attention, and the cache's write and
read, against plain implementations.

Tables are whole numbers and equal.  The norm: everything is fp32, with sums over at most 128 terms
and a handful of roundings a value: within 1e-5 of the sizes of the terms a value is the sum of;
bf16 outputs add half a step, 2^-8 of the value at most.  Cached values are the nearest of their block's
MXFP4 form; where a value's fp32 error (1e-5 of its size) reaches over the border between two codes,
or the largest of a block over a power of two, either form is right."""
from __future__ import annotations

import numpy as np
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


def _i(v, dtype=I32):
    return torch.tensor(np.asarray(v), dtype=dtype, device="cuda")


# ---- tables --------------------------------------------------------------------------------


def _tables64(held, new, free, at, end, table, page, tokens):
    table, F = table.copy(), len(free)
    starts, slots, pos = [0], [], []
    for b, (h, n) in enumerate(zip(held, new)):
        for i in range(-(-h // page), -(-(h + n) // page)):
            table[b, i] = free[at % F]
            at += 1
        for p in range(h, h + n):
            slots.append(table[b, p // page] * page + p % page)
            pos.append(p)
        starts.append(starts[-1] + n)
    assert at <= end
    pad = tokens - len(slots)
    return table, np.add(held, new), starts, slots + [-1] * pad, pos + [0] * pad, at


def _make(B, page, most_held, most_new, seed, columns=2):
    g = np.random.default_rng(seed)
    held, new = g.integers(0, most_held + 1, B), g.integers(0, most_new + 1, B)
    if B > 2:
        held[1], new[2] = 0, 0
    had, want = -(-held // page), -(-(held + new) // page)
    ids = g.permutation(int(want.sum()) + 9) if B else np.arange(9)
    table = np.full((B, (int(want.max()) if B else 0) + columns), -7, np.int64)
    at = 0
    for b in range(B):
        table[b, :had[b]] = ids[at:at + had[b]]
        at += had[b]
    return held, new, table, ids[at:]


def _call(held, new, table, free, at, end, page, tokens, status=None, in_place=False):
    B = len(held)
    d = dict(held=_i(held), new_tokens=_i(new), free_pages=_i(free), free_range=_i([at, end], torch.int64),
             page=page, table=_i(table), starts=_i(np.full(B + 1, 77)), slots=_i(np.full(tokens, 77)),
             positions=_i(np.full(tokens, 77)))
    d["lengths"] = d["held"] if in_place else _i(np.full(B, 77))
    d["free_out"] = d["free_range"] if in_place else _i([77, 77], torch.int64)
    moe.cache_tables(**d, status=status)
    return {k: v.cpu().numpy() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


@pytest.mark.parametrize("B,page,held,new,spare", [
    (1, 16, 0, 1, 0), (1, 64, 63, 1, 0), (3, 16, 40, 5, 3), (8, 128, 9000, 1, 7), (33, 32, 300, 40, 100),
    (1000, 16, 200, 3, 1), (1025, 64, 4000, 30, 12), (16384, 16, 20, 2, 5), (5, 16, 100000, 30000, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(lib, B, page, held, new, spare, in_place):
    held, new, table, free = _make(B, page, held, new, seed=B)
    turn = 3 % len(free)
    tokens = int(new.sum()) + spare
    base = 5 * len(free)   # `next` counts on beyond the ring's size
    got = _call(held, new, table, np.roll(free, turn), base + turn, base + turn + len(free), page, tokens,
                in_place=in_place)
    want = _tables64(held, new, np.roll(free, turn), base + turn, base + turn + len(free), table, page, tokens)
    for name, w in zip(("table", "lengths", "starts", "slots", "positions"), want):
        assert np.array_equal(got[name], w), name
    assert list(got["free_out"]) == [want[5], base + turn + len(free)]


def test_tables_of_no_requests_and_no_tokens(lib):
    got = _call([], [], np.zeros((0, 4), np.int64), [1, 2], 0, 2, 16, 5)
    assert list(got["starts"]) == [0] and list(got["slots"]) == [-1] * 5 and list(got["free_out"]) == [0, 2]
    got = _call([16, 3], [0, 0], np.array([[4, 9], [5, 9]]), [1], 0, 1, 16, 0)
    assert list(got["lengths"]) == [16, 3] and list(got["starts"]) == [0, 0, 0]


@pytest.mark.parametrize("what", ["pages", "columns", "rows", "held", "new", "id", "range"])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_step_that_does_not_fit_is_not_made(lib, what, in_place):
    """All or nothing: the status word says why, and every output is an empty step's."""
    held, new, page = np.array([20, 0, 33]), np.array([13, 16, 4]), 16
    table, free = np.array([[3, 4, -7, -7], [-7] * 4, [8, 9, 10, -7]]), np.arange(20, 30)
    at, end, tokens, bit = 2, 10, 40, moe.DEV_NO_ROOM
    if what == "pages":
        end = 3
    elif what == "columns":
        table = table[:, :2].copy()
    elif what == "rows":
        tokens = 32
    elif what == "range":
        end = 13   # more than the ring has
    else:
        bit = moe.DEV_BAD_INDEX
        if what == "held":
            held[1] = -1
        elif what == "new":
            new[2] = -3
        else:
            table[2, 2] = -1   # the page that request 2's next token joins
    status = _i([0])
    got = _call(held, new, table, free, at, end, page, tokens, status, in_place)
    assert int(status) & bit
    assert np.array_equal(got["lengths"], held) and np.array_equal(got["table"], table)
    assert not got["starts"].any() and not got["positions"].any() and (got["slots"] == -1).all()
    assert list(got["free_out"]) == [at, end]


def test_tables_step_after_step_in_a_graph(lib):
    """Replays of one captured call, in place, are the steps of one call after the other."""
    B, page, F = 4, 16, 40
    held, table = _i([0, 15, 16, 31]), _i(np.full((B, 12), -7))
    table[1, 0], table[2, 0], table[3, 0], table[3, 1] = 100, 101, 102, 103
    new, free = _i([1, 2, 1, 3]), _i(np.arange(F))
    span = _i([0, F], torch.int64)
    starts, slots, pos = _i(np.zeros(B + 1)), _i(np.zeros(9)), _i(np.zeros(9))
    state = [t.clone() for t in (held, table, span)]
    args = (new, free, span, page, table, held, starts, slots, pos, span)
    moe.cache_tables(held, *args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.cache_tables(held, *args)
    for t, s in zip((held, table, span), state):
        t.copy_(s)
    h, tb, at = np.array([0, 15, 16, 31]), state[1].cpu().numpy(), 0
    for _ in range(20):
        g.replay()
        tb, h, st, sl, ps, at = _tables64(h, new.tolist(), list(range(F)), at, F, tb, page, 9)
        assert held.tolist() == list(h) and slots.tolist() == sl and pos.tolist() == ps
        assert span.tolist() == [at, F] and np.array_equal(table.cpu().numpy(), tb)


# ---- norm, rotation, cache -------------------------------------------------------------------


def _rope64(qkv, pos, cs, Hq, Hk, D, w_q, w_k, eps, pairs):
    """(q, k, v, sizes of q's and k's terms) in fp64."""
    x = qkv[:, :(Hq + 2 * Hk) * D].double().reshape(-1, Hq + 2 * Hk, D)
    out = []
    for part, w in ((x[:, :Hq], w_q), (x[:, Hq:Hq + Hk], w_k)):
        if w is not None:
            part = part / torch.sqrt((part * part).mean(-1, keepdim=True) + eps) * w.double()
        size = part.abs().clone()
        part = part.clone()
        if cs is not None:
            R = cs.shape[1]
            t = cs.double()[pos.long()][:, None]
            cos, sin = t[..., :R // 2], t[..., R // 2:]
            i = torch.arange(0, R, 2) if pairs else torch.arange(R // 2)
            j = i + 1 if pairs else i + R // 2
            a, b = part[..., i], part[..., j]
            part[..., i], part[..., j] = a * cos - b * sin, b * cos + a * sin
            size[..., i] = size[..., j] = (a * a + b * b).sqrt() * 2
        out.append((part, size))
    return out[0][0], out[1][0], x[:, Hq + Hk:], out[0][1], out[1][1]


def _close_bf16(got, ref, size):
    bound = 1e-5 * (ref.abs() + size) + ref.abs() * 2 ** -8
    assert bool(((got.double() - ref).abs() <= bound).all()), float(((got.double() - ref).abs() / bound).max())


def _inputs(T, Hq, Hk, D, R, param, stride=None, far=1000, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    width = (Hq + 2 * Hk) * D
    rows = (r(T, stride or width) * 2).bfloat16()
    qkv = rows[:, :width] if stride else rows
    pos = torch.randint(0, far, (T,), device="cuda", generator=g, dtype=I32)
    cs = moe.rope_table(far, R) if R else None
    w = [None if param is None else (1 + 0.1 * r(D)).to(param) for _ in range(2)]
    return qkv, pos, cs, w[0], w[1]


SHAPES = [(1, 1, 1, 64, 64), (1, 64, 8, 128, 128), (7, 64, 8, 128, 128), (3, 5, 5, 128, 64), (5, 12, 3, 64, 32),
          (300, 8, 2, 128, 16), (2, 7, 1, 64, 0), (33, 40, 8, 128, 128), (5000, 6, 2, 64, 48), (700, 64, 8, 128, 96)]


@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("param", [None, BF, torch.float32])
def test_rope(lib, T, Hq, Hk, D, R, style, param):
    qkv, pos, cs, wq, wk = _inputs(T, Hq, Hk, D, R, param, stride=(Hq + 2 * Hk) * D + 24)
    q, k = torch.empty(T, Hq, D, dtype=BF, device="cuda"), torch.empty(T, Hk, D, dtype=BF, device="cuda")
    moe.qk_norm_rope(qkv, pos, cs, Hq, Hk, q, k_out=k, w_q=wq, w_k=wk, eps=1e-5, style=style)
    q64, k64, _, sq, sk = _rope64(qkv, pos, cs, Hq, Hk, D, wq, wk, 1e-5, style == 1)
    _close_bf16(q, q64, sq)
    _close_bf16(k, k64, sk)


def _nearest(v):
    c, s = mx4.quantize(v.cpu().numpy())
    return torch.tensor(mx4.dequantize(c, s), device=v.device)


@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
@pytest.mark.parametrize("style,page", [(0, 16), (1, 64)])
def test_cache_write_and_read(lib, T, Hq, Hk, D, R, style, page):
    qkv, pos, cs, wq, wk = _inputs(T, Hq, Hk, D, R, BF, seed=1)
    pages = -(-T // page) + 2
    g = torch.Generator(device="cuda").manual_seed(2)
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:T].to(I32)
    if T > 2:
        slots[T // 2] = -1
    cache = moe.Cache4(pages, page, Hk, D)
    cache.codes.fill_(0x5a), cache.scales.fill_(0xc3)
    before = cache.codes.clone(), cache.scales.clone()
    bf = dict(dtype=BF, device="cuda")
    q, q2, k = torch.empty(T, Hq, D, **bf), torch.empty(T, Hq, D, **bf), torch.empty(T, Hk, D, **bf)
    status = _i([0])
    moe.qk_norm_rope(qkv, pos, cs, Hq, Hk, q, w_q=wq, w_k=wk, style=style, cache=cache, slots=slots, status=status)
    moe.qk_norm_rope(qkv, pos, cs, Hq, Hk, q2, k_out=k, w_q=wq, w_k=wk, style=style, cache=cache, slots=slots,
                     status=status)
    assert torch.equal(q, q2) and int(status) == 0
    # nothing else in the cache has changed
    there = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    there[slots[slots >= 0].long()] = True
    there = there.reshape(pages, 1, 1, page)
    for now, old in zip((cache.codes, cache.scales), before):
        assert torch.equal(now[~there.expand(pages, 2, Hk, page)], old[~there.expand(pages, 2, Hk, page)])
    ck, cv = torch.full((T, Hk, D), 9.0, **bf), torch.full((T, Hk, D), 9.0, **bf)
    moe.cache_read(cache, slots, ck, cv, status=status)
    assert int(status) == 0
    kept = (slots >= 0)
    assert bool((ck[~kept] == 9).all()) and bool((cv[~kept] == 9).all())   # left as they were
    _, k64, v64, _, sk = _rope64(qkv, pos, cs, Hq, Hk, D, wq, wk, 1e-6, style == 1)
    assert torch.equal(cv[kept].double(), _nearest(v64[kept]))          # values as they are: no error at all
    lo, hi = _nearest(k64[kept] - 1e-5 * sk[kept]), _nearest(k64[kept] + 1e-5 * sk[kept])
    mid, got = _nearest(k64[kept]), ck[kept].double()
    off = got != mid
    assert float(off.double().mean()) < 1e-3
    assert bool(((got == mid) | (got == lo) | (got == hi)).all())
    one = torch.empty_like(cv)
    moe.cache_read(cache, slots[kept], v=one[:int(kept.sum())])          # either alone
    assert torch.equal(one[:int(kept.sum())], cv[kept])


def test_cache_holds_what_mx4_quantize_gives(lib):
    """The same codes and scale bytes, also of blocks with an infinity, a NaN, zeros and tiny numbers."""
    T, Hk, D, page = 20, 3, 128, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(T, 7 * D, device="cuda", generator=g).bfloat16()
    qkv[1, 5 * D] = float("inf")
    qkv[2, 6 * D + 40] = float("nan")
    qkv[3, 4 * D:] = 0
    qkv[4, 4 * D:] *= 1e-38
    qkv[5, 4 * D:] *= 1e38
    cache, q = moe.Cache4(2, page, Hk, D), torch.empty(T, 1, D, dtype=BF, device="cuda")
    slots = torch.arange(T, device="cuda", dtype=I32) + 5
    moe.qk_norm_rope(qkv, None, None, 1, Hk, q, cache=cache, slots=slots)
    codes, scales = moe.mx4_quantize(qkv[:, D:].reshape(T, 2, Hk, D).contiguous())
    at = slots.long()
    assert torch.equal(cache.codes[at // page, :, :, at % page], codes)
    assert torch.equal(cache.scales[at // page, :, :, at % page], scales)
    assert torch.equal(q[:, 0], qkv[:, :D])


def test_rows_whose_place_is_outside_are_not_written(lib):
    T, D = 6, 64
    qkv, pos, cs, wq, wk = _inputs(T, 2, 1, D, D, BF, far=50)
    pos[1], pos[4] = -1, 50
    slots = _i([0, 1, 32, 3, 4, -2])
    cache = moe.Cache4(2, 16, 1, D)
    cache.codes.fill_(7), cache.scales.fill_(7)
    q = torch.full((T, 2, D), 5.0, dtype=BF, device="cuda")
    status = _i([0])
    moe.qk_norm_rope(qkv, pos, cs, 2, 1, q, w_q=wq, w_k=wk, cache=cache, slots=slots, status=status)
    assert int(status) == moe.DEV_BAD_INDEX
    for t in (1, 2, 4, 5):
        assert bool((q[t] == 5).all())
    assert bool((cache.codes[0, :, :, 1] == 7).all()) and bool((cache.codes[0, :, :, 4] == 7).all())
    assert bool((cache.codes[1] == 7).all())
    q64, _, _, sq, _ = _rope64(qkv[[0, 3]], pos[[0, 3]], cs, 2, 1, D, wq, wk, 1e-6, False)
    _close_bf16(q[[0, 3]], q64, sq)
    status.zero_()
    k = torch.full((3, 1, D), 5.0, dtype=BF, device="cuda")
    moe.cache_read(cache, _i([32, -2, 0]), k, status=status)
    assert int(status) == moe.DEV_BAD_INDEX and bool((k[:2] == 5).all()) and not bool((k[2] == 5).all())


def test_zero_and_non_finite_heads(lib):
    T, D = 4, 128
    qkv, pos, cs, wq, wk = _inputs(T, 2, 1, D, D, torch.float32)
    qkv[0, :D] = 0
    qkv[1, 5] = float("nan")
    qkv[2, 7] = float("inf")
    q, k = torch.empty(T, 2, D, dtype=BF, device="cuda"), torch.empty(T, 1, D, dtype=BF, device="cuda")
    moe.qk_norm_rope(qkv, pos, cs, 2, 1, q, k_out=k, w_q=wq, w_k=wk)
    assert not bool(q[0, 0].any()) and bool(torch.isnan(q[1, 0]).all()) and bool(torch.isnan(q[2, 0]).any())
    good = torch.ones(T, 2, dtype=torch.bool, device="cuda")
    good[1, 0] = good[2, 0] = False
    q64, k64, _, sq, sk = _rope64(qkv, pos, cs, 2, 1, D, wq, wk, 1e-6, False)
    _close_bf16(q[good], q64[good], sq[good])
    _close_bf16(k, k64, sk)


def test_no_rows(lib):
    z = torch.empty(0, 4 * 64, dtype=BF, device="cuda")
    moe.qk_norm_rope(z, _i([]), moe.rope_table(4, 64), 2, 1, torch.empty(0, 2, 64, dtype=BF, device="cuda"),
                     k_out=torch.empty(0, 1, 64, dtype=BF, device="cuda"))
    moe.cache_read(moe.Cache4(1, 16, 1, 64), _i([]), torch.empty(0, 1, 64, dtype=BF, device="cuda"))
