"""Norm and rotation of rows that lie in larger tensors: one row of any width, rows more than 2^31 elements apart."""
from __future__ import annotations

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from _gpu_common import build_library

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _call(qkv, T, Hq=2, Hk=1, D=64):
    q, k = torch.zeros(T, Hq, D, dtype=BF, device="cuda"), torch.zeros(T, Hk, D, dtype=BF, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    moe.qk_norm_rope(qkv, pos, moe.rope_table(8, 32), Hq, Hk, q, k)
    return q, k


@pytest.mark.parametrize("more", [0, 1, 3, 8, 13])
def test_one_row_of_any_width(lib, more):
    """What one row gives does not depend on how many columns lie behind its heads."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.randn(2, 256 + 16, device="cuda", generator=g).bfloat16()
    want = _call(rows[:, :256], 2)
    for got, w in zip(_call(rows[:1, :256 + more], 1), want):
        assert torch.equal(got, w[:1])


def test_rows_further_apart_than_a_stride_can_say_are_refused(lib):
    """2^32 + 256 elements: in 32 bits that would be 256, rows of another place."""
    far = 2 ** 32 + 256
    qkv = torch.empty(far + 256, dtype=BF, device="cuda").as_strided((2, 256), (far, 1))
    with pytest.raises(ValueError):
        _call(qkv, 2)
