"""What the binding refuses of the tensors of a call: each of these would be read or written out of
its bounds, or as another type."""
from __future__ import annotations

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


def _empty(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_product_tensors(lib):
    G, N, K, R = 3, 256, 384, 10
    good = dict(a=_empty(R, K // 2), a_scales=_empty(R, K // 32), w=_empty(G, N, K // 2),
                w_scales=_empty(G, N, K // 32), c=_empty(R, N, dtype=torch.float32),
                expert_offsets=torch.tensor([0, 2, 2, R], dtype=torch.int32, device="cuda"),
                status=_empty(1, dtype=torch.int32))

    def call(kind=moe.OUT_F32, rows=R, **kw):
        v = {**good, **kw}
        moe.mx4_grouped_gemm(G, N, K, rows, v["a"], v["a_scales"], v["expert_offsets"], v["w"],
                             v["w_scales"], v["c"], kind, v["status"])
    call()
    call(a=_empty(R + 3, K // 2), c=_empty(R + 1, N, dtype=torch.float32))   # more rows than used
    call(status=None, expert_offsets=good["expert_offsets"].data_ptr())
    call(c=good["c"].bfloat16(), kind=moe.OUT_BF16)
    for name, bad in (
            ("a", good["a"][:-1]), ("a", good["a"].int()), ("a", good["a"].cpu()),
            ("a", _empty(R, K)), ("a", _empty(K // 2, R).t()), ("a_scales", good["a_scales"][:-1]),
            ("a_scales", _empty(R, K // 16)), ("w", good["w"][:-1]), ("w", _empty(G * 2, N // 2, K // 2)),
            ("w_scales", good["w_scales"][1:]), ("w_scales", _empty(G, N, K // 32, dtype=torch.int32)),
            ("c", good["c"][:-1]), ("c", good["c"].bfloat16()), ("c", good["c"].half()),
            ("expert_offsets", good["expert_offsets"][:-1]), ("expert_offsets", good["expert_offsets"].long()),
            ("status", _empty(1))):
        with pytest.raises((TypeError, ValueError)):
            call(**{name: bad})
    with pytest.raises((TypeError, ValueError)):
        call(kind=moe.OUT_BF16)
    with pytest.raises(moe.MoEError):
        call(kind=9)
    with pytest.raises(moe.MoEError):
        call(a=None)
    call(rows=0, a=None)


def test_swiglu_tensors(lib):
    G, I, K, R = 2, 128, 256, 5
    off = torch.tensor([0, 2, R], dtype=torch.int32, device="cuda")
    good = dict(h=_empty(R, I // 2), h_scales=_empty(R, I // 32), w13=_empty(G, 2 * I, K // 2))

    def call(**kw):
        v = {**good, **kw}
        moe.mx4_grouped_gemm_swiglu(G, I, K, R, _empty(R, K // 2), _empty(R, K // 32), off, v["w13"],
                                    _empty(G, 2 * I, K // 32), v["h"], v["h_scales"])
    call()
    for name, bad in (("h", _empty(R, I)), ("h", good["h"][1:]), ("h_scales", good["h_scales"].int()),
                      ("h_scales", good["h_scales"][:-1]), ("w13", good["w13"][:, :I].contiguous())):
        with pytest.raises((TypeError, ValueError)):
            call(**{name: bad})
