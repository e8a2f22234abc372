"""What the binding refuses before the library is called (no GPU needed)."""
from __future__ import annotations

import dataclasses

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
import synth
from moe_expert_layer_07_gb300 import ep

MX4 = synth.MoEShape("four bits", tokens=4, hidden=256, inter=128, num_experts=4, num_shared=1,
                     top_k=2, dtype="mxfp4")


def _codes(shape):
    G, H, I = shape.groups, shape.hidden, shape.inter
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    return dict(wg=torch.zeros(shape.num_experts, H, dtype=torch.bfloat16), w13=u8(G, 2 * I, H // 2),
                w13_s=u8(G, 2 * I, H // 32), w2=u8(G, H, I // 2), w2_s=u8(G, H, I // 32))


def test_layers_of_other_types_refuse_mxfp4():
    """Four-bit codes are not read as bf16 rows of twice their size."""
    with pytest.raises(ValueError):
        moe.MoELayer(MX4, _codes(MX4))
    with pytest.raises(ValueError):
        moe.MoELayer(MX4, _codes(MX4), pack_weights=False)
    plan = ep.EPPlan(MX4.num_experts, 1, 0)
    with pytest.raises(ValueError):
        ep.GpuRank(MX4, _codes(MX4), plan)


def test_packing_refuses_elements_of_another_size():
    w = torch.zeros(2, 128, 128, dtype=torch.uint8)
    for dtype in ("bf16", "fp8"):
        cfg = moe.make_config(dataclasses.replace(MX4, dtype=dtype))
        good = w if dtype == "fp8" else w.bfloat16()
        for bad in (good.float(), w if dtype == "bf16" else w.bfloat16()):
            with pytest.raises(TypeError):
                moe.pack_expert_weights(cfg, bad)
        with pytest.raises(TypeError):
            moe.pack_expert_weights(cfg, good, out=good[:1])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_the_mxfp4_layer_refuses_other_types(dtype):
    """It took them up to 16 tokens, and read their bytes as codes above."""
    with pytest.raises(ValueError):
        moe.Mx4MoELayer(dataclasses.replace(MX4, dtype=dtype), _codes(MX4), 40)
    with pytest.raises(TypeError):
        moe.Mx4MoELayer(MX4, object(), 40)


def test_few_token_layer_refuses_weights_of_another_size():
    four = dataclasses.replace(MX4, dtype="bf16")
    for shape, w in ((four, _codes(MX4)), (dataclasses.replace(MX4, dtype="fp8"), _codes(MX4)),
                     (MX4, dict(_codes(MX4), w2=None))):
        with pytest.raises((TypeError, ValueError)):
            moe.FewTokenLayer(shape, w)
