"""The few-token layer.

Routing: ids and weights equal moe_route's, bit for bit.  The rest in two steps, so that a value
of h on a rounding boundary cannot hide an error or make one: (1) each stored h against fp64,
where it may be further from it than the nearest value of its format by 2e-5 of its block's (BF16: its
128 features') largest (fp32 sums of at most 7168 products, a fast exponential and division); (2) the output
against fp64 sums over the h that was stored, within 5e-5 of the output's rms (fp32 sums of at
most 2048 exact products, and of at most 20 rows)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_expert_layer_07_gb300 as moe
import synth
from oracle import mx4

from _gpu_common import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _shape(T, H, I, E, S, k, dtype, scoring="softmax", groups=1, norm=True, scaling=1.0):
    return synth.MoEShape("few", tokens=T, hidden=H, inter=I, num_experts=E, num_shared=S, top_k=k,
                          num_groups=groups, topk_groups=max(1, groups // 2), group_topn=min(2, E // groups),
                          scoring=scoring, norm_topk=norm, routed_scaling=scaling, dtype=dtype,
                          bias_std=0.01 if scoring == "sigmoid" else None)


def _inputs(shape, seed=0):
    """Device tensors, and the expert weights' values in fp64 (a function of the group)."""
    if shape.dtype != "mxfp4":
        w = synth.make_inputs(shape, seed=seed, device="cuda")
    else:
        import dataclasses
        w = synth.make_inputs(dataclasses.replace(shape, dtype="bf16"), seed=seed, device="cuda")
        for key in ("w13", "w2"):
            w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
    if w["x"].shape[0] != shape.tokens:
        raise AssertionError

    def values(key, g):
        if shape.dtype == "bf16":
            return w[key][g].double()
        if shape.dtype == "fp8":
            s = w[key + "_s"][g].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            return w[key][g].view(torch.float8_e4m3fn).double() * s
        return torch.tensor(mx4.dequantize(w[key][g].cpu().numpy(), w[key + "_s"][g].cpu().numpy()),
                            device="cuda")
    return w, values


def _x_values(shape, x):
    if shape.dtype == "bf16":
        return x.double()
    if shape.dtype == "mxfp4":
        return torch.tensor(mx4.dequantize(*mx4.quantize(x.cpu().double().numpy())), device="cuda")
    T, H = x.shape
    b = x.float().view(T, H // 128, 128)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return ((b / s).to(torch.float8_e4m3fn).double() * s.double()).view(T, H)


def _nearest_error(shape, h):
    """|nearest value of h's format - h| and the largest |h| of its block, per element."""
    n = 32 if shape.dtype == "mxfp4" else 128
    b = h.view(h.shape[0], -1, n)
    amax = b.abs().amax(-1, keepdim=True).expand_as(b).reshape(h.shape)
    if shape.dtype == "bf16":
        hi = h.bfloat16().double()   # two parts
        return (hi + (h - hi).bfloat16().double() - h).abs(), amax
    if shape.dtype == "mxfp4":
        v = torch.tensor(mx4.dequantize(*mx4.quantize(h.cpu().numpy())), device="cuda")
        return (v - h).abs(), amax
    s = b.abs().amax(-1, keepdim=True).clamp(min=1e-300) / 448.0
    v = ((b / s).float().to(torch.float8_e4m3fn).double() * s).view(h.shape)
    return (v - h).abs(), amax


def _stored_h(shape, layer, R):
    I = shape.inter
    if shape.dtype == "bf16":
        return layer.view("h", torch.bfloat16, (R, I // 64, 2, 64)).double().sum(2).reshape(R, I)
    if shape.dtype == "fp8":   # segments of 128 values: fp16 code values, then the fp32 scale
        seg = layer.view("h", torch.uint8, (R, I // 128, 272))
        v = seg[..., :256].contiguous().view(torch.float16).double()
        return (v * seg[..., 256:260].contiguous().view(torch.float32).double()).reshape(R, I)
    codes = layer.view("h", torch.uint8, (R, I // 2)).cpu().numpy()
    most = layer.cfg.max_tokens * (shape.top_k + shape.num_shared) + 16
    s = layer.view("h_scales", torch.uint8, (I // 128, most, 16))[:, :R, :4]
    s = s.permute(1, 0, 2).reshape(R, I // 32).cpu().numpy()
    return torch.tensor(mx4.dequantize(codes, s), device="cuda")


def _check(shape, w, values, layer, out_dtype=torch.float32, T=None, log2phys=None):
    T = shape.tokens if T is None else T
    x = w["x"][:T].contiguous()
    k, E, S, H = shape.top_k, shape.num_experts, shape.num_shared, shape.hidden
    out = torch.full((T, H), float("nan"), dtype=out_dtype, device="cuda")
    layer.forward(x, out, moe.OUT_F32 if out_dtype == torch.float32 else moe.OUT_BF16)
    assert layer.status() == 0
    # routing
    cfg = moe.make_config(shape, T)
    cfg.dtype = moe.BF16
    logits = torch.empty(T, E, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, k, device="cuda")
    moe.route(cfg, T, x, w["wg"], w.get("e_bias"), w.get("logit_offset"), log2phys, logits, ids, tw)
    assert torch.equal(layer.view("topk_ids", torch.int32, (T, k)), ids)
    assert torch.equal(layer.view("topk_w", torch.float32, (T, k)), tw)
    # h and the output, group by group
    xq = _x_values(shape, x)
    nid, nw = ids.cpu().numpy(), tw.double()
    R = T * (k + S)
    hs = _stored_h(shape, layer, R)
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    row = 0
    for g in list(range(E, E + S)) + sorted(set(nid.reshape(-1).tolist())):
        toks = list(range(T)) if g >= E else [t for t in range(T) if g in nid[t]]
        tk = torch.tensor(toks, device="cuda")
        o = xq[tk] @ values("w13", g).t()
        gate, up = o[:, :shape.inter], o[:, shape.inter:]
        h = gate / (1 + torch.exp(-gate)) * up
        got = hs[row:row + len(toks)]
        near, amax = _nearest_error(shape, h)
        off = (got - h).abs() - near
        assert float((off - 2e-5 * amax).max()) <= 0, (g, float((off / amax.clamp(min=1e-30)).max()))
        wt = torch.ones(len(toks), 1, dtype=torch.float64, device="cuda")
        if g < E:
            wt = torch.stack([nw[t, list(nid[t]).index(g)] for t in toks])[:, None]
        ref[tk] += wt * (got @ values("w2", g).t())
        row += len(toks)
    assert row == R
    rms = float(ref.square().mean().sqrt())
    bound = 5e-5 * rms
    if out_dtype == torch.bfloat16:   # half a unit in the last place
        bound = bound + torch.exp2(torch.frexp(ref)[1].double() - 9)
    assert bool(((out.double() - ref).abs() <= bound).all()), \
        (float((out.double() - ref).abs().max()), rms)
    return out


DTYPES = ["bf16", "fp8", "mxfp4"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 15, 16])
def test_tokens(lib, dtype, T):
    s = _shape(T, 1024, 384, 32, 1, 8, dtype, scoring="sigmoid", groups=8, scaling=2.5)
    w, v = _inputs(s, T)
    _check(s, w, v, moe.FewTokenLayer(s, w))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,I", [(128, 128), (128, 2048), (2048, 1408), (7168, 256), (384, 640)])
def test_sizes(lib, dtype, H, I):
    s = _shape(3, H, I, 8, 2, 3, dtype)
    w, v = _inputs(s, H + I)
    _check(s, w, v, moe.FewTokenLayer(s, w), torch.bfloat16)


@pytest.mark.parametrize("E,S,k,scoring,groups,norm",
                         [(1, 0, 1, "softmax", 1, True), (4, 0, 4, "softmax", 1, False),
                          (16, 4, 1, "sigmoid", 1, False), (60, 0, 16, "sigmoid", 2, True),
                          (200, 1, 6, "softmax", 1, True), (512, 0, 8, "sigmoid", 8, True),
                          (1024, 1, 2, "softmax", 1, False)])
def test_routings(lib, E, S, k, scoring, groups, norm):
    s = _shape(13, 256, 128, E, S, k, "fp8", scoring=scoring, groups=groups, norm=norm)
    w, v = _inputs(s, E)
    _check(s, w, v, moe.FewTokenLayer(s, w))


@pytest.mark.parametrize("dtype", ["fp8", "mxfp4"])
def test_full_width(lib, dtype):
    s = _shape(16, 7168, 2048, 16, 1, 8, dtype, scoring="sigmoid", groups=8, scaling=2.5)
    w, v = _inputs(s, 5)
    _check(s, w, v, moe.FewTokenLayer(s, w), torch.bfloat16)


def test_one_expert_takes_every_token(lib):
    """All tokens on the same experts: groups of 16 rows, the others empty."""
    s = _shape(16, 512, 256, 8, 0, 2, "bf16")
    w, v = _inputs(s)
    w["x"][:] = w["x"][0]
    out = _check(s, w, v, moe.FewTokenLayer(s, w))
    assert bool((out == out[0]).all())


def test_permutation_offsets_and_shared_layer_weights(lib):
    """log2phys and logit_offset; weights shared with an MoELayer (packed once)."""
    s = _shape(6, 512, 256, 16, 1, 4, "fp8", scoring="sigmoid", groups=4)
    w, v = _inputs(s, 3)
    w["logit_offset"] = torch.linspace(-1, 1, 16, device="cuda")
    l2p = torch.randperm(16, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    big = moe.MoELayer(s, w, log2phys=l2p)
    few = moe.FewTokenLayer(s, big)
    out = _check(s, w, v, few, log2phys=l2p.cuda())
    ref = torch.empty_like(out)
    big.forward(w["x"], ref)
    # the layer's own tolerance: h may differ by a code where it lies on a boundary
    assert float((out - ref).abs().max()) <= 2e-2 * float(ref.square().mean().sqrt())


@pytest.mark.parametrize("dtype", DTYPES)
def test_repeatable_and_independent_of_the_workspace(lib, dtype):
    s = _shape(16, 1024, 512, 32, 1, 8, dtype)
    w, v = _inputs(s, 7)
    layer = moe.FewTokenLayer(s, w)
    layer.ws.fill_(0xFF)
    a = torch.empty(16, 1024, device="cuda")
    layer.forward(w["x"], a)
    for _ in range(20):
        b = torch.empty_like(a)
        layer.forward(w["x"], b)
        assert torch.equal(a, b)
    # fewer tokens in the same workspace, then as before
    c = torch.empty(3, 1024, device="cuda")
    layer.forward(w["x"][:3].contiguous(), c)
    layer.forward(w["x"], b)
    assert torch.equal(a, b) and layer.status() == 0


def test_graph_capture_and_other_stream(lib):
    s = _shape(4, 512, 256, 16, 1, 4, "fp8", scoring="sigmoid")
    w, v = _inputs(s, 2)
    layer = moe.FewTokenLayer(s, w)
    a, b = torch.empty(4, 512, device="cuda"), torch.empty(4, 512, device="cuda")
    layer.forward(w["x"], a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer.forward(w["x"], b)
        with torch.cuda.graph(g, stream=side):
            layer.forward(w["x"], b)
    b.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_no_tokens_and_invalid_ids(lib):
    s = _shape(4, 256, 128, 8, 1, 2, "bf16")
    w, v = _inputs(s, 4)
    layer = moe.FewTokenLayer(s, w)
    layer.forward(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"),
                  torch.empty(0, 256, device="cuda"))
    assert layer.status() == 0
    # a permutation table with ids out of range: the status word says so, and the output is the
    # shared expert's alone (or zeros without one)
    for S in (1, 0):
        s = _shape(4, 256, 128, 8, S, 2, "bf16")
        w, v = _inputs(s, 4)
        layer = moe.FewTokenLayer(s, w, log2phys=[99] * 8)
        out = torch.full((4, 256), float("nan"), device="cuda")
        layer.forward(w["x"], out)
        assert layer.status() == moe.DEV_BAD_EXPERT_ID
        ref = torch.zeros(4, 256, dtype=torch.float64, device="cuda")
        if S:
            o = w["x"].double() @ v("w13", 8).t()
            h = (o[:, :128] / (1 + torch.exp(-o[:, :128])) * o[:, 128:])
            ref = h @ v("w2", 8).t()
            assert float((out.double() - ref).abs().max()) <= 1e-2 * float(ref.square().mean().sqrt())
        else:
            assert not out.any()


def test_non_finite_tokens_stay_their_own(lib):
    """A token with an infinity or a NaN leaves the others' outputs as they were."""
    s = _shape(5, 256, 128, 8, 1, 2, "mxfp4")
    w, v = _inputs(s, 9)
    layer = moe.FewTokenLayer(s, w)
    a, b = torch.empty(5, 256, device="cuda"), torch.empty(5, 256, device="cuda")
    layer.forward(w["x"], a)
    w["x"][1, 17] = float("inf")
    w["x"][3, 5] = float("nan")
    layer.forward(w["x"], b)
    for t in (0, 2, 4):
        assert torch.equal(a[t], b[t])
    assert bool(torch.isnan(b[1]).all()) and bool(torch.isnan(b[3]).all())


def test_refusals(lib):
    s = _shape(4, 256, 128, 8, 1, 2, "bf16")
    w, _ = _inputs(s)
    x, out = w["x"], torch.empty(4, 256, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.FewTokenLayer(s, w, max_tokens=17)
    layer = moe.FewTokenLayer(s, w, max_tokens=3)
    with pytest.raises(moe.MoEError):
        layer.forward(x, out)                      # more tokens than the workspace is for
    with pytest.raises(moe.MoEError):
        layer.forward(x[:2], out[:2], out_dtype=9)
    with pytest.raises(moe.MoEError):
        moe.layer_few(layer.cfg, layer.weights, 2, x, out, moe.OUT_F32, layer.ws, layer.ws_bytes - 1)
    layer.weights.expert_layout = moe.LAYOUT_ROWS
    with pytest.raises(moe.MoEError):              # expert weights that are not packed
        layer.forward(x[:2], out[:2])
    with pytest.raises(ValueError):
        moe.FewTokenLayer(s, moe.MoELayer(s, w, pack_weights=False))
