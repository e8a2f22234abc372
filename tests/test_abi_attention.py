"""The entry points of attention over the four-bit cache on the host (no GPU needed): every refusal
comes before any launch, sizes are what the header says, and the binding refuses unsuitable tensors."""
import ctypes

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from moe_expert_layer_07_gb300 import attention as A

P = ctypes.c_void_p
FAKE, ODD = P(0x1000), P(0x1008)   # never dereferenced


@pytest.fixture(scope="module")
def L():
    from moe_expert_layer_07_gb300 import _build
    _build.build()
    return moe.lib()


def _cache(**kw):
    d = dict(codes=0x1000, scales=0x1000, pages=8, kv_heads=2, page=16, dim=128)
    d.update(kw)
    return A._Cache(**d)


BAD_CACHES = [(dict(dim=96), -2), (dict(page=8), -2), (dict(page=48), -2), (dict(kv_heads=257), -2),
              (dict(kv_heads=0), -1), (dict(pages=-1), -1), (dict(codes=None), -1), (dict(scales=0x1008), -1),
              (dict(pages=1 << 27, page=16), -2)]


def test_tables_refusals(L):
    names = ("held", "new", "free", "range", "table", "lengths", "starts", "slots", "positions", "out")

    def call(B=3, page=16, count=4, columns=5, tokens=6, **kw):
        p = {n: FAKE for n in names}
        p.update(kw)
        return L.moe_cache_tables(B, page, p["held"], p["new"], p["free"], count, p["range"], p["table"],
                                  columns, p["lengths"], p["starts"], p["slots"], p["positions"], tokens,
                                  p["out"], None, None)
    assert call(B=-1) == -1 and call(count=-1) == -1 and call(columns=-1) == -1 and call(tokens=-1) == -1
    assert call(page=0) == -1 and call(page=8) == -2 and call(page=256) == -2 and call(page=24) == -2
    assert call(B=16385) == -2
    for n in names:
        assert call(**{n: None}) == -1, n
        assert call(**{n: ODD}) == -1, n


def test_rope_refusals(L):
    def call(T=2, qkv=FAKE, pos=FAKE, cs=FAKE, wq=FAKE, wk=FAKE, q=FAKE, k=FAKE, cache=None, slots=None, **kw):
        d = dict(q_heads=4, kv_heads=2, dim=128, rope_dim=128, style=0, param_dtype=1, max_positions=10,
                 qkv_stride=1024, eps=1e-6)
        d.update(kw)
        return L.moe_qk_norm_rope(A._Rope(**d), T, qkv, pos, cs, wq, wk, q, k, cache, slots, None, None)
    assert call(T=0, qkv=None) == 0
    assert L.moe_qk_norm_rope(None, 2, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, None, None, None, None) == -1
    assert call(T=-1) == -1 and call(q_heads=0) == -1 and call(kv_heads=0) == -1 and call(dim=0) == -1
    assert call(style=2) == -1 and call(param_dtype=2) == -1 and call(eps=-1.0) == -1 and call(eps=float("nan")) == -1
    assert call(dim=96) == -2 and call(rope_dim=24) == -2 and call(rope_dim=144) == -2 and call(qkv_stride=1028) == -2
    assert call(qkv_stride=1016) == -1                        # shorter than the heads
    assert call(max_positions=0) == -1 and call(pos=None) == -1 and call(cs=None) == -1
    assert call(k=None) == -1                                 # keys to nowhere
    assert call(slots=FAKE) == -1 and call(cache=_cache()) == -1
    assert call(cache=_cache(dim=64), slots=FAKE) == -1 and call(cache=_cache(kv_heads=4), slots=FAKE) == -1
    for bad, rc in BAD_CACHES:
        assert call(cache=_cache(**bad), slots=FAKE) == rc, bad
    for name in ("qkv", "q"):
        assert call(**{name: None}) == -1, name
    for name in ("qkv", "pos", "cs", "wq", "wk", "q", "k"):
        assert call(**{name: ODD}) == -1, name
    assert call(cache=_cache(), slots=ODD) == -1


def test_read_refusals(L):
    def call(n=2, slots=FAKE, k=FAKE, v=FAKE, **kw):
        return L.moe_cache_read(_cache(**kw), n, slots, k, v, None, None)
    assert call(n=0, slots=None) == 0 and call(n=-1) == -1
    assert call(slots=None) == -1 and call(k=None, v=None) == -1
    assert call(slots=ODD) == -1 and call(k=ODD) == -1 and call(v=ODD) == -1
    for bad, rc in BAD_CACHES:
        assert call(**bad) == rc, bad


def test_attention_refusals(L):
    def desc(**kw):
        d = dict(requests=2, rows=3, q_heads=4, max_pages=4, max_q=2, max_len=64, window=0, scale=0.1)
        d.update(kw)
        return A._Attn(**d)
    n = ctypes.c_size_t()
    size = lambda d, c: L.moe_cache_attention_workspace_size(d, c, ctypes.byref(n))  # noqa: E731
    assert size(desc(), _cache()) == 0
    need = n.value
    assert need > 0 and need % 256 == 0

    def call(q=FAKE, table=FAKE, lengths=FAKE, starts=FAKE, out=P(0x9000), kind=1, lse=None, ws=FAKE, nb=need,
             cache=None, **kw):
        return L.moe_cache_attention(desc(**kw), cache or _cache(), q, table, lengths, starts, out, kind, lse, ws,
                                     nb, None, None)
    assert call(requests=0, q=None) == 0 and call(rows=0, q=None) == 0
    for bad in (dict(requests=-1), dict(rows=-1), dict(q_heads=0), dict(max_pages=-1), dict(max_q=-1),
                dict(max_len=-1), dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**bad) == -1, bad
        assert size(desc(**bad), _cache()) == -1, bad
    assert call(requests=4097) == -2 and call(q_heads=5) == -2 and call(rows=1 << 30) == -2
    for bad, rc in BAD_CACHES:
        assert call(cache=_cache(**bad)) == rc, bad
        assert size(desc(), _cache(**bad)) == rc, bad
    for name in ("q", "table", "lengths", "starts", "out", "ws"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -1, name
    assert call(lse=ODD) == -1 and call(kind=2) == -1
    assert call(out=FAKE, kind=0) == -1                       # in place, of another type
    assert call(nb=need - 1) == -3
    assert L.moe_cache_attention_workspace_size(desc(), _cache(), None) == -1
    assert L.moe_cache_attention_workspace_size(None, _cache(), ctypes.byref(n)) == -1


def test_w4_refusals(L):
    def call(T=2, x=FAKE, w=FAKE, s=FAKE, z=None, y=FAKE, kind_out=0, **kw):
        d = dict(n_out=64, k_dim=256, kind=0, group=32, scale_dtype=0)
        d.update(kw)
        return L.moe_w4_matvec(A._W4(**d), T, x, w, s, z, y, kind_out, None)
    assert call(T=0, x=None) == 0 and call(T=-1) == -1 and call(T=17) == -2
    assert L.moe_w4_matvec(None, 2, FAKE, FAKE, FAKE, None, FAKE, 0, None) == -1
    assert call(n_out=0) == -1 and call(k_dim=0) == -1 and call(kind=2) == -1 and call(kind_out=2) == -1
    assert call(group=64) == -2 and call(kind=1, group=48) == -2 and call(k_dim=272) == -2 and call(k_dim=32800) == -2
    assert call(kind=1, group=128, k_dim=320) == -2 and call(kind=1, scale_dtype=3) == -1
    assert call(z=FAKE) == -1                                 # MXFP4 has no zero points
    for name in ("x", "w", "s", "y"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -1, name
    assert call(kind=1, z=ODD) == -1


def test_w4_refuses_more_columns_than_its_counts_hold(L):
    d = A._W4(n_out=(1 << 30) + 1, k_dim=32, kind=0, group=32, scale_dtype=0)
    assert L.moe_w4_matvec(d, 1, FAKE, FAKE, FAKE, None, FAKE, 0, None) == -2


def test_binding_refuses_wrong_tensors():
    """Shapes, types and places: a tensor on the CPU is not passed on either."""
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    with pytest.raises(ValueError):
        moe.Cache4(4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        moe.Cache4.of(torch.zeros(4, 2, 16, 32, dtype=u8), torch.zeros(4, 2, 16, 2, dtype=u8))
    with pytest.raises(TypeError):
        moe.Cache4.of(torch.zeros(4, 2, 1, 16, 32), torch.zeros(4, 2, 1, 16, 2))
    i = lambda *s: torch.zeros(*s, dtype=i32)  # noqa: E731
    good = dict(held=i(3), new_tokens=i(3), free_pages=i(4), free_range=torch.zeros(2, dtype=torch.int64), page=16,
                table=i(3, 5), lengths=i(3), starts=i(4), slots=i(6), positions=i(6),
                free_out=torch.zeros(2, dtype=torch.int64))
    for bad in ({}, dict(held=i(3).long()), dict(starts=i(3)), dict(table=i(2, 5)), dict(positions=i(5)),
                dict(free_range=i(2)), dict(table=i(5, 3).t())):
        with pytest.raises((TypeError, ValueError)):
            moe.cache_tables(**{**good, **bad})
    qkv, q = torch.zeros(2, 8 * 64, dtype=bf), torch.zeros(2, 4, 64, dtype=bf)
    for bad in ({}, dict(qkv=qkv.float()), dict(q_out=q.float()), dict(qkv=qkv[:, :100]), dict(q_out=q[:1]),
                dict(w_q=q[0, 0].half()), dict(slots=i(2))):
        args = dict(qkv=qkv, positions=None, cos_sin=None, q_heads=4, kv_heads=2, q_out=q)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            moe.qk_norm_rope(**args)
    x, w = torch.zeros(2, 64, dtype=bf), torch.zeros(8, 32, dtype=u8)
    s, y = torch.zeros(8, 2, dtype=u8), torch.zeros(2, 8)
    for bad in ({}, dict(x=x.float()), dict(codes=w.int()), dict(scales=s.int()), dict(out=y.half()),
                dict(out=y[:1]), dict(scales=s[:, :0]), dict(zeros=s), dict(codes=w[:, :16])):
        with pytest.raises((TypeError, ValueError)):
            moe.w4_matvec(**{**dict(x=x, codes=w, scales=s, out=y), **bad})


def test_rope_table_is_rounded_once():
    import math
    t = moe.rope_table(100001, 16, base=10000.0, device="cpu")
    assert t.dtype is torch.float32 and t.shape == (100001, 16)
    for pos, i in ((0, 0), (100000, 0), (99999, 3), (100000, 7)):
        a = pos * 10000.0 ** (-2 * i / 16)
        assert abs(float(t[pos, i]) - math.cos(a)) < 2 ** -24 and abs(float(t[pos, 8 + i]) - math.sin(a)) < 2 ** -24
