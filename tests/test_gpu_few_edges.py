"""The few-token layer where its tables and numbers are unusual."""
from __future__ import annotations

import dataclasses

import pytest
import torch

import moe_expert_layer_07_gb300 as moe
import synth

from _gpu_common import build_library

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "fp8", "mxfp4"]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _inputs(shape, seed=0):
    four = shape.dtype == "mxfp4"
    w = synth.make_inputs(dataclasses.replace(shape, dtype="bf16") if four else shape, seed=seed,
                          device="cuda")
    if four:
        for key in ("w13", "w2"):
            w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
    return w


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k,table", [
    (1, 8, 3, [5] * 8),                       # one token's choices all on one slot
    (3, 8, 2, [0, 0, 1, 1, 2, 2, 3, 3]),      # pairs of experts on a slot
    (8, 8, 2, [7] * 8),                       # 16 rows of one expert, 8 to a group
    (9, 16, 4, [2] * 12 + [15, 14, 13, 13]),
    (16, 16, 16, [3] * 16),                   # as many rows of one expert as there can be
    (16, 16, 16, [1, 0] * 8)])
def test_experts_that_share_a_slot(lib, dtype, T, E, k, table):
    """log2phys may name a slot more than once: the same bits as with the slots' weights written out
    for each logical expert, since a row's products do not depend on the rows beside it."""
    s = synth.MoEShape("shared slots", tokens=T, hidden=384, inter=256, num_experts=E, num_shared=1,
                       top_k=k, dtype=dtype)
    w = _inputs(s, T + k)
    few = moe.FewTokenLayer(s, w, log2phys=table)
    few.ws[4:].fill_(0xFF)
    got = torch.full((T, 384), float("nan"), device="cuda")
    few.forward(w["x"], got)
    assert few.status() == 0
    at = torch.tensor(table + [E], device="cuda")
    spread = dict(w, **{key: w[key][at].contiguous() for key in ("w13", "w13_s", "w2", "w2_s")
                        if w[key] is not None})
    ref = torch.empty_like(got)
    moe.FewTokenLayer(s, spread).forward(w["x"], ref)
    assert torch.equal(got, ref)
    ids = few.view("topk_ids", torch.int32, (T, k))
    assert bool((ids[..., None] == at[:E].int()).any(-1).all())


@pytest.mark.parametrize("T", [4, 40])
def test_status_of_the_mxfp4_layer_is_the_last_calls(lib, T):
    """A token of NaN has no expert to go to; the next call starts anew, on each path and after
    either."""
    shape = synth.MoEShape("status", tokens=40, hidden=256, inter=128, num_experts=8, num_shared=1,
                           top_k=2, dtype="mxfp4")
    w = _inputs(shape)
    layer = moe.Mx4MoELayer(shape, w, 40)
    assert layer.status() == 0
    x, out = w["x"], torch.empty(40, 256, device="cuda")
    bad = x.clone()
    bad[1] = float("nan")
    layer.ids.zero_()
    for after in (4, 40):
        layer.forward(bad[:T], out[:T])
        assert layer.status() == moe.DEV_BAD_EXPERT_ID
        layer.forward(x[:after], out[:after])
        assert layer.status() == 0
        layer.forward(bad[:after], out[:after])
        layer.forward(x[:T], out[:T])
        assert layer.status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer.forward(bad[:T], out[:T], stream=side)
    side.synchronize()
    assert layer.status() == moe.DEV_BAD_EXPERT_ID
    layer.forward(x[:T], out[:T], stream=side.cuda_stream)
    side.synchronize()
    assert layer.status() == 0


def test_an_overflowing_h_stays_an_infinity(lib):
    """h beyond bf16's range: the few-token layer, which keeps h in two parts, answers as the layer
    does.  Token 0's h overflows fp32, token 1's lies between the largest bf16 and the largest fp32
    number, token 2's is NaN, token 3's an ordinary one."""
    s = synth.MoEShape("large h", tokens=4, hidden=256, inter=128, num_experts=4, num_shared=0, top_k=1,
                       dtype="bf16")
    w = _inputs(s, 1)
    w["wg"].zero_()
    w["wg"][torch.arange(4), torch.arange(4)] = 1.0       # token t to expert t
    w["x"].zero_()
    w["x"][torch.arange(4), torch.arange(4)] = 1.0
    w["w13"].zero_()
    w["w13"][0, :128, 0], w["w13"][0, 128:, 0] = 1e19, 1e20       # h beyond fp32 too
    w["x"][1, 10] = 1.0                                            # 2^64 (0.9961 + 0.0030) 2^64
    w["w13"][1, :128, 1], w["w13"][1, 128:, 1], w["w13"][1, 128:, 10] = 2.0 ** 64, 1.8374687e19, 5.534e16
    w["w13"][2, :128, 2], w["w13"][2, 128:, 2] = float("inf"), 0.0
    w["w13"][3, :128, 3], w["w13"][3, 128:, 3] = 3.0, 5.0
    w["w2"][:2] = w["w2"][:2].abs() + 0.01
    big = moe.MoELayer(s, w)
    few = moe.FewTokenLayer(s, big)
    ref, got = torch.empty(4, 256, device="cuda"), torch.empty(4, 256, device="cuda")
    big.forward(w["x"], ref)
    few.forward(w["x"], got)
    assert few.status() == big.status() == 0
    assert bool((ref[:2] == float("inf")).all()) and torch.equal(got[:2], ref[:2])
    assert bool(torch.isnan(got[2]).all())
    assert bool(torch.isfinite(got[3]).all()) and float((got[3] - ref[3]).abs().max()) <= 2e-2 * float(ref[3].abs().max())


def _route(s, w):
    """moe_route's (ids, weights, status)."""
    cfg = moe.make_config(s, s.tokens)
    dev = dict(device="cuda")
    ids = torch.full((s.tokens, s.top_k), -1, dtype=torch.int32, **dev)
    tw, st = torch.zeros(s.tokens, s.top_k, **dev), torch.zeros(1, dtype=torch.int32, **dev)
    moe.route(cfg, s.tokens, w["x"], w["wg"], w["e_bias"], None, None,
              torch.empty(s.tokens, s.num_experts, **dev), ids, tw, st)
    return ids, tw, int(st)


# live experts of each group, the others' bias is minus infinity
@pytest.mark.parametrize("live", [[16, 16, 1, 1], [16, 1, 0, 1], [2, 1, 1, 0], [1, 1, 1, 1], [0, 0, 3, 0],
                                  [0, 0, 0, 0], [16, 3, 2, 2]])
@pytest.mark.parametrize("gs", [16, 32, 64])
@pytest.mark.parametrize("topn", [1, 2, 4, 5])
@pytest.mark.parametrize("keep,k", [(2, 2), (3, 1), (4, 4)])
def test_routing_with_experts_taken_out(lib, live, gs, topn, keep, k):
    """A bias of minus infinity takes an expert out of the selection; the groups that are kept, the ids,
    the weights and what is reported are moe_route's."""
    s = synth.MoEShape("masked", tokens=5, hidden=128, inter=128, num_experts=4 * gs, num_shared=0,
                       top_k=k, num_groups=4, topk_groups=keep, group_topn=topn, scoring="sigmoid",
                       norm_topk=True, routed_scaling=2.5, dtype="bf16", bias_std=0.01)
    w = _inputs(s, gs)
    bias = torch.full((4, gs), float("-inf"), device="cuda")
    for g, n in enumerate(live):
        # groups of few live experts have the best ones, which only the group's score keeps out
        bias[g, gs // 2 - n // 2:gs // 2 - n // 2 + n] = 0.01 if n == 16 else 1.0
    w["e_bias"] = bias.reshape(-1).contiguous()
    ids, tw, st = _route(s, w)
    few = moe.FewTokenLayer(s, w)
    few.forward(w["x"], torch.empty(5, 128, device="cuda"))
    assert few.status() == st
    assert torch.equal(few.view("topk_ids", torch.int32, (5, k)), ids)
    assert torch.equal(few.view("topk_w", torch.float32, (5, k)), tw)
