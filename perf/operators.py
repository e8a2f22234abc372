"""What is measured of the operators around the MoE layer: the few-token layer, MXFP4
quantisation and its grouped products, and the norms around a block.

Each case names one operator and its sizes.  ``run`` computes it either in plain fp32 torch
operations or, with ``own`` set, by the library's entry points; ``exact`` computes it in fp64.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32          # elements that share one MXFP4 scale
FEW = 16            # most tokens of a few-token call

# ---- cases ---------------------------------------------------------------------------

_TINY = dict(hidden=1024, inter=512, experts=16, shared=1, top_k=4, num_groups=1, topk_groups=1,
             group_topn=1, scoring="softmax", norm=True, scaling=1.0)
_V2 = dict(hidden=2048, inter=1408, experts=64, shared=2, top_k=6, num_groups=1, topk_groups=1,
           group_topn=1, scoring="softmax", norm=False, scaling=1.0)
_R1 = dict(hidden=7168, inter=2048, experts=256, shared=1, top_k=8, num_groups=8, topk_groups=4,
           group_topn=2, scoring="sigmoid", norm=True, scaling=2.5)


def listed():
    return [
        # one user's next token through the smallest layer: launches and waits are most of it
        dict(name="few_tiny_bf16_t1", op="few", dtype="bf16", tokens=1, **_TINY),
        # five requests decoding together, BF16 experts of an odd width, two shared experts
        dict(name="few_v2lite_bf16_t5", op="few", dtype="bf16", tokens=5, **_V2),
        # one request on the 256-expert FP8 layer: nine experts' weights read for one row each
        dict(name="few_r1_fp8_t1", op="few", dtype="fp8", tokens=1, **_R1),
        # the most tokens of a call, as in a small server's step or a draft's verification
        dict(name="few_r1_fp8_t16", op="few", dtype="fp8", tokens=16, **_R1),
        # the same layer with its experts in four bits, three requests
        dict(name="few_r1_mxfp4_t3", op="few", dtype="mxfp4", tokens=3, **_R1),
        # activations of a decode step quantised and read back: two short launches
        dict(name="mx4_quant_t24", op="quant", rows=24, cols=7168, dtype="bf16"),
        # activations of a long prompt
        dict(name="mx4_quant_t16384", op="quant", rows=16384, cols=7168, dtype="bf16"),
        # down products of a decode step: a few rows for each expert, weights are all of it
        dict(name="mx4_gemm_decode", op="gemm", groups=33, rows=273, n=7168, k=2048),
        # gate and up products with SwiGLU of a prompt over 32 experts, uneven groups
        dict(name="mx4_swiglu_prompt", op="swiglu", groups=33, rows=4599, n=2048, k=7168),
        # down products of a long prompt: the tensor cores' own rate
        dict(name="mx4_gemm_long", op="gemm", groups=8, rows=16411, n=7168, k=2048),
        # the norms around a block, one decode step of seven tokens
        dict(name="norm_t7", op="norm", tokens=7, hidden=7168, kind="rms", y="fp32", res="bf16",
             post=True, pre=True, gate="none", alpha=1.0, beta=1.0),
        # a long prompt, gated by feature and scaled as deep networks do
        dict(name="norm_t16384", op="norm", tokens=16384, hidden=7168, kind="rms", y="bf16",
             res="bf16", post=True, pre=True, gate="feature", alpha=0.9, beta=0.35),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _multiple(rng, unit, lo, hi):
    v = unit * _log_int(rng, lo, hi)
    return v + unit if v == 3072 else v   # a size that no configuration here has


def draw(rng):
    op = rng.choice(["few", "few", "quant", "gemm", "swiglu", "norm"])
    if op == "few":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log_int(rng, 4, 32)
        topk_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, topk_groups * (experts // groups)))
        scoring = rng.choice(["softmax", "sigmoid"])
        return dict(op="few", dtype=rng.choice(["bf16", "fp8", "mxfp4"]), tokens=_log_int(rng, 1, FEW),
                    hidden=_multiple(rng, 128, 2, 56), inter=_multiple(rng, 128, 1, 16),
                    experts=experts, shared=rng.randint(0, 2), top_k=top_k, num_groups=groups,
                    topk_groups=topk_groups, group_topn=rng.randint(1, 2), scoring=scoring,
                    norm=rng.random() < 0.5, scaling=rng.choice([1.0, 2.5]))
    if op == "quant":
        return dict(op="quant", rows=_log_int(rng, 1, 16384), cols=_multiple(rng, BLOCK, 1, 224),
                    dtype=rng.choice(["bf16", "fp32"]))
    if op == "gemm":
        return dict(op="gemm", groups=_log_int(rng, 1, 48), rows=_log_int(rng, 1, 16384),
                    n=_multiple(rng, 128, 1, 56), k=_multiple(rng, 128, 1, 16))
    if op == "swiglu":
        return dict(op="swiglu", groups=_log_int(rng, 1, 33), rows=_log_int(rng, 1, 4096),
                    n=_multiple(rng, 128, 1, 16), k=_multiple(rng, 128, 1, 56))
    return dict(op="norm", tokens=_log_int(rng, 1, 16384), hidden=_multiple(rng, 8, 16, 896),
                kind=rng.choice(["rms", "layer"]), y=rng.choice(["bf16", "fp32"]),
                res=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.7, pre=rng.random() < 0.8,
                gate=rng.choice(["none", "feature", "token", "full"]),
                alpha=rng.choice([1.0, 0.8]), beta=rng.choice([1.0, 0.25]))


# ---- MXFP4, FP8 and routing in plain operations ---------------------------------------

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power(byte):
    """2^(byte - 127) in fp32, from its bits (0 stands for 2^-127, a subnormal number)."""
    b = byte.int()
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _mx4_split(v):
    """v fp32 [..., n] -> (magnitude's code, sign, scale byte) of blocks of 32: the scale's
    exponent is floor(log2(amax)) - 2 (0 for a block of zeros), values round to nearest even."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    byte = torch.where(amax > 0, (torch.frexp(amax)[1] + 124).clamp(min=0), 127)
    a = b.abs() / _power(byte)
    idx = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
           + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    return idx, (b < 0), byte


def _mx4_round(v):
    """The values that v's MXFP4 form stands for."""
    idx, neg, byte = _mx4_split(v)
    mag = torch.tensor(_E2M1, dtype=v.dtype, device=v.device)[idx.long()]
    return (torch.where(neg, -mag, mag) * _power(byte)).reshape(v.shape)


def _mx4_pack(v):
    """v [..., n] -> codes uint8 [..., n/2] (even element in the low half), scales uint8
    [..., n/32] (exponent + 127)."""
    idx, neg, byte = _mx4_split(v)
    c = (idx + 8 * neg.int()).reshape(*v.shape[:-1], -1, 2)
    codes = (c[..., 0] + 16 * c[..., 1]).to(torch.uint8)
    return codes, byte[..., 0].to(torch.uint8)


def _mx4_values(codes, scales):
    """codes uint8 [..., n/2], scales uint8 [..., n/32] -> fp32 values [..., n]."""
    table = torch.tensor(_E2M1 + tuple(-m for m in _E2M1), device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], dim=-1)
    v = table[both.int()].reshape(*scales.shape, BLOCK)
    return (v * _power(scales).unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _fp8_round(v):
    """The values that v's FP8 form (e4m3, one scale amax / 448 for 128 columns) stands for."""
    b = v.reshape(*v.shape[:-1], -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    # a tensor as divisor: by a number torch multiplies with the reciprocal
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    q = (b / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return (q.float() * s).reshape(v.shape)


def _fp8_values(codes, scales):
    """codes e4m3 [..., N, K], scales [..., N/128, K/128] -> fp32 values."""
    n, k = codes.shape[-2:]
    v = codes.float().reshape(*codes.shape[:-2], n // 128, 128, k // 128, 128)
    return (v * scales[..., :, None, :, None]).reshape(codes.shape)


def _activation(v, dtype):
    return {"bf16": lambda t: t, "fp8": _fp8_round, "mxfp4": _mx4_round}[dtype](v)


def _route(c, logits, bias):
    """(ids [T, k], weights [T, k]) of the layer's routing; ties go to the lowest index."""
    T, E = logits.shape
    score = torch.sigmoid(logits) if c["scoring"] == "sigmoid" else logits
    sel = score + bias if bias is not None else score
    if c["num_groups"] > 1:
        per = sel.reshape(T, c["num_groups"], -1)
        gscore = per.sort(-1, descending=True)[0][..., :c["group_topn"]].sum(-1)
        kept = gscore.sort(dim=-1, descending=True, stable=True)[1][:, :c["topk_groups"]]
        mask = torch.zeros(T, c["num_groups"], dtype=torch.bool, device=sel.device)
        mask.scatter_(1, kept, True)
        sel = torch.where(mask.unsqueeze(-1), per, torch.full_like(per, -math.inf)).reshape(T, E)
    ids = sel.sort(dim=-1, descending=True, stable=True)[1][:, :c["top_k"]]
    if c["scoring"] == "sigmoid":
        w = score.gather(1, ids)
    else:
        w = torch.exp(logits - logits.amax(-1, keepdim=True))
        w = (w if c["norm"] else w / w.sum(-1, keepdim=True)).gather(1, ids)
    if c["norm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids, w * c["scaling"]


def _normed(v, kind, eps, w, b):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * w
    return n if b is None else n + b


# ---- inputs ------------------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    v = torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)
    return (v * scale).to(dtype)


def _few_shape(c):
    import synth
    return synth.MoEShape("few", tokens=c["tokens"], hidden=c["hidden"], inter=c["inter"],
                          num_experts=c["experts"], num_shared=c["shared"], top_k=c["top_k"],
                          num_groups=c["num_groups"], topk_groups=c["topk_groups"],
                          group_topn=c["group_topn"], scoring=c["scoring"], norm_topk=c["norm"],
                          routed_scaling=c["scaling"], dtype=c["dtype"])


def _offsets(c, seed):
    """Rows of each group: uneven, the first of three or more groups empty."""
    g = np.random.default_rng(seed)
    p = g.gamma(4.0, size=c["groups"])
    if c["groups"] >= 3:
        p[0] = 0.0
    return np.concatenate([[0], np.cumsum(g.multinomial(c["rows"], p / p.sum()))])


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if own:
        import moe_expert_layer_07_gb300 as moe
        s["moe"] = moe
    if c["op"] == "few":
        G, H, I = c["experts"] + c["shared"], c["hidden"], c["inter"]
        s["x"] = _randn(gen, c["tokens"], H, dtype=torch.bfloat16)
        s["wg"] = _randn(gen, c["experts"], H, dtype=torch.bfloat16, scale=0.02)
        s["e_bias"] = _randn(gen, c["experts"], scale=0.01) if c["scoring"] == "sigmoid" else None
        for key, n, k in (("w13", 2 * I, H), ("w2", H, I)):
            if c["dtype"] == "bf16":
                s[key] = torch.empty(G, n, k, dtype=torch.bfloat16, device="cuda")
            elif c["dtype"] == "fp8":
                s[key] = torch.empty(G, n, k, dtype=torch.float8_e4m3fn, device="cuda")
                s[key + "_s"] = torch.empty(G, n // 128, k // 128, device="cuda")
            else:
                s[key] = torch.empty(G, n, k // 2, dtype=torch.uint8, device="cuda")
                s[key + "_s"] = torch.empty(G, n, k // BLOCK, dtype=torch.uint8, device="cuda")
            for g in range(G):   # one expert at a time: the fp32 values of all would not fit
                v = _randn(gen, n, k, scale=0.02)
                if c["dtype"] == "bf16":
                    s[key][g] = v
                elif c["dtype"] == "fp8":
                    b = v.reshape(n // 128, 128, k // 128, 128)
                    sc = b.abs().amax((1, 3)) / 448.0
                    s[key + "_s"][g] = sc
                    s[key][g] = (b / sc[:, None, :, None]).reshape(n, k).to(torch.float8_e4m3fn)
                else:
                    s[key][g], s[key + "_s"][g] = _mx4_pack(v)
        if own:
            s["layer"] = s["moe"].FewTokenLayer(_few_shape(c), s)
            s["out"] = torch.empty(c["tokens"], H, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "quant":
        # rows of different sizes, as a residual stream's are
        s["x"] = _randn(gen, c["rows"], c["cols"])
        s["x"] = (s["x"] * torch.exp(_randn(gen, c["rows"], 1))).to(_TYPES[c["dtype"]])
        if own:
            s["codes"] = torch.empty(c["rows"], c["cols"] // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(c["rows"], c["cols"] // BLOCK, dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty(c["rows"], c["cols"], dtype=torch.bfloat16, device="cuda")
    elif c["op"] in ("gemm", "swiglu"):
        n = c["n"] * (2 if c["op"] == "swiglu" else 1)
        off = _offsets(c, seed)
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        s["most"] = int(np.diff(off).max())
        s["a"], s["a_s"] = _mx4_pack(_randn(gen, c["rows"], c["k"]))
        s["w"] = torch.empty(c["groups"], n, c["k"] // 2, dtype=torch.uint8, device="cuda")
        s["w_s"] = torch.empty(c["groups"], n, c["k"] // BLOCK, dtype=torch.uint8, device="cuda")
        for g in range(c["groups"]):
            s["w"][g], s["w_s"][g] = _mx4_pack(_randn(gen, n, c["k"], scale=0.02))
        if own:
            s["wt"], s["wt_s"] = s["moe"].pack_mx4_weights(s["w"], s["w_s"])
            s["out"] = torch.empty(c["rows"], c["n"], dtype=torch.bfloat16, device="cuda")
            if c["op"] == "swiglu":
                s["h"] = torch.empty(c["rows"], c["n"] // 2, dtype=torch.uint8, device="cuda")
                s["h_s"] = torch.empty(c["rows"], c["n"] // BLOCK, dtype=torch.uint8, device="cuda")
    else:
        T, H = c["tokens"], c["hidden"]
        s["y"] = _randn(gen, T, H, dtype=_TYPES[c["y"]], scale=0.5)
        s["res"] = _randn(gen, T, H, dtype=_TYPES[c["res"]], scale=3.0)
        for key in ("post", "pre"):
            on = c[key]
            s["w_" + key] = (1 + _randn(gen, H, scale=0.1)).bfloat16() if on else None
            s["b_" + key] = _randn(gen, H, dtype=torch.bfloat16, scale=0.1) \
                if on and c["kind"] == "layer" else None
        gshape = {"none": None, "feature": (H,), "token": (T,), "full": (T, H)}[c["gate"]]
        s["gate"] = None if gshape is None else _randn(gen, *gshape, dtype=torch.bfloat16)
        if own:
            s["res_out"] = torch.empty_like(s["res"])
            s["x_out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda") if c["pre"] else None
    return s


# ---- one pass ------------------------------------------------------------------------------


def _expert_values(s, key, ids):
    """The weights of the experts ids [...], as fp32 values [..., N, K]."""
    kind = s["case"]["dtype"]
    if kind == "bf16":
        return s[key][ids].float()
    if kind == "fp8":
        codes = s[key].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
        return _fp8_values(codes, s[key + "_s"][ids])
    return _mx4_values(s[key][ids], s[key + "_s"][ids])


def _plain_few(s):
    c, x = s["case"], s["x"].float()
    ids, w = _route(c, x @ s["wg"].float().t(), s["e_bias"])
    T = x.shape[0]
    shared = torch.arange(c["experts"], c["experts"] + c["shared"], device=x.device)
    ids = torch.cat([ids, shared.expand(T, -1)], 1)
    w = torch.cat([w, torch.ones(T, c["shared"], device=x.device)], 1)
    xq = _activation(x, c["dtype"])
    gu = torch.matmul(_expert_values(s, "w13", ids), xq[:, None, :, None])[..., 0]
    g, u = gu.split(c["inter"], dim=-1)
    h = _activation(g * torch.sigmoid(g) * u, c["dtype"])
    y = torch.matmul(_expert_values(s, "w2", ids), h.unsqueeze(-1))[..., 0]
    return (y * w.unsqueeze(-1)).sum(1).bfloat16()


def _plain_gemm(s):
    c, off = s["case"], s["offsets"].long()
    a = _mx4_values(s["a"], s["a_s"])
    w = _mx4_values(s["w"], s["w_s"])
    row = torch.arange(c["rows"], device=a.device)
    group = torch.searchsorted(off[1:], row, right=True)
    at = row - off[group]
    padded = a.new_zeros(c["groups"], s["most"], c["k"])
    padded[group, at] = a
    out = torch.bmm(padded, w.transpose(1, 2))[group, at]
    if c["op"] == "swiglu":
        g, u = out.split(c["n"], dim=-1)
        out = _mx4_round(g * torch.sigmoid(g) * u)
    return out.bfloat16()


def _norm_formula(s, dtype):
    c = s["case"]
    as_ = lambda t: None if t is None else t.to(dtype)  # noqa: E731
    n = as_(s["y"])
    if c["post"]:
        n = _normed(n, c["kind"], 1e-6, as_(s["w_post"]), as_(s["b_post"]))
    if s["gate"] is not None:
        n = n * (as_(s["gate"]).unsqueeze(-1) if c["gate"] == "token" else as_(s["gate"]))
    r = c["alpha"] * as_(s["res"]) + c["beta"] * n
    x = _normed(r, c["kind"], 1e-6, as_(s["w_pre"]), as_(s["b_pre"])) if c["pre"] else None
    return r, x


def run(state):
    s, c = state, state["case"]
    if own:
        moe = s["moe"]
        if c["op"] == "few":
            return s["layer"].forward(s["x"], s["out"], moe.OUT_BF16)
        if c["op"] == "quant":
            moe.mx4_quantize(s["x"], s["codes"], s["scales"])
            return moe.mx4_dequantize(s["codes"], s["scales"], s["out"])
        if c["op"] == "gemm":
            moe.mx4_grouped_gemm(c["groups"], c["n"], c["k"], c["rows"], s["a"], s["a_s"],
                                 s["offsets"], s["wt"], s["wt_s"], s["out"], moe.OUT_BF16)
            return s["out"]
        if c["op"] == "swiglu":
            moe.mx4_grouped_gemm_swiglu(c["groups"], c["n"], c["k"], c["rows"], s["a"], s["a_s"],
                                        s["offsets"], s["wt"], s["wt_s"], s["h"], s["h_s"])
            return moe.mx4_dequantize(s["h"], s["h_s"], s["out"])
        moe.block_norm(s["res"], y=s["y"], residual_out=s["res_out"], x_out=s["x_out"],
                       w_post=s["w_post"], b_post=s["b_post"], w_pre=s["w_pre"],
                       b_pre=s["b_pre"], gate=s["gate"], residual_scale=c["alpha"],
                       branch_scale=c["beta"], eps=1e-6,
                       kind=moe.NORM_LAYER if c["kind"] == "layer" else moe.NORM_RMS)
        return {"residual": s["res_out"], "x": s["x_out"]}
    if c["op"] == "few":
        return _plain_few(s)
    if c["op"] == "quant":
        return _mx4_round(s["x"].float()).bfloat16()
    if c["op"] in ("gemm", "swiglu"):
        return _plain_gemm(s)
    r, x = _norm_formula(s, torch.float32)
    return {"residual": r.to(_TYPES[c["res"]]), "x": None if x is None else x.bfloat16()}


# ---- what a pass cannot do without -----------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "few":
        T, E, k, H, I = c["tokens"], c["experts"], c["top_k"], c["hidden"], c["inter"]
        # experts with at least one row, expected for independent uniform choices
        active = E * (1.0 - (1.0 - k / E) ** T) + c["shared"]
        per = {"bf16": 2.0, "fp8": 1.0 + 4.0 / 16384, "mxfp4": 0.5 + 1.0 / BLOCK}[c["dtype"]]
        return {"bytes": active * 3 * H * I * per + 2 * E * H + 4 * T * H,
                "flops": 2.0 * T * (E * H + (k + c["shared"]) * 3 * H * I)}
    if c["op"] == "quant":
        n = c["rows"] * c["cols"]
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": n * (size + 2 + 2 * (0.5 + 1.0 / BLOCK)), "flops": 4.0 * n}
    if c["op"] in ("gemm", "swiglu"):
        G, R, n, k = c["groups"], c["rows"], c["n"], c["k"]
        wide = n * (2 if c["op"] == "swiglu" else 1)
        # groups that hold a row: the first of three or more is empty
        full = min(R, G - 1 if G >= 3 else G)
        bits = 0.5 + 1.0 / BLOCK
        out = R * n * (2 if c["op"] == "gemm" else 2 * bits + 2)
        return {"bytes": full * wide * k * bits + R * k * bits + out, "flops": 2.0 * R * wide * k}
    T, H = c["tokens"], c["hidden"]
    size = {"bf16": 2, "fp32": 4}
    gate = {"none": 0, "feature": 2 * H, "token": 2 * T, "full": 2 * T * H}[c["gate"]]
    return {"bytes": T * H * (size[c["y"]] + 2 * size[c["res"]] + (2 if c["pre"] else 0)) + gate
            + 2 * H * (c["post"] + c["pre"]) * (2 if c["kind"] == "layer" else 1),
            "flops": 10.0 * T * H}


# ---- the definition in 64 bits ----------------------------------------------------------------


def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e2m1_64(v):
    """v fp64 [..., n]: each block of 32 over its power of two, the nearest of the fifteen values
    (ties: the one whose code is even), times that power."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    top = b.abs().max(-1, keepdim=True)[0]
    p = _power64((torch.frexp(top)[1] - 3).clamp(min=-127))
    p = torch.where(top > 0, p, torch.ones_like(p))
    r = b / p
    a = r.abs().clamp(max=6.0)
    # the step between neighbours is 1/2 below 2, 1 below 4 and 2 above; round() ties to even
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.copysign(torch.round(a / step) * step, r) * p).reshape(v.shape)


def _e4m3_64(v):
    """The layer's FP8 form of v fp64.  Its definition takes the scale and the quotients in fp32
    (quotients of bf16 values often lie midway between two codes, and that decides them)."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 128, 128).float()
    top = b.abs().max(-1, keepdim=True)[0]
    p = torch.where(top > 0, torch.div(top, torch.tensor(448.0, device=v.device).expand_as(top)),
                    torch.ones_like(top))
    r = (b / p).double()
    a = r.abs().clamp(max=448.0)
    # three mantissa bits, the smallest normal 2^-6
    step = _power64((torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
    return (torch.copysign(torch.round(a / step) * step, r) * p.double()).reshape(v.shape)


def _mx4_64(codes, scales):
    """Values in fp64 from the bits: sign, two exponent bits (bias 1), one mantissa bit."""
    nib = torch.stack([codes.long() & 15, codes.long() >> 4], -1).flatten(-2)
    ex, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * _power64(ex - 1))
    val = torch.where(nib >= 8, -mag, mag)
    return val * _power64(scales.long() - 127).repeat_interleave(BLOCK, -1)


def _silu64(g):
    return g / (1.0 + torch.exp(-g))


def exact(case, seed):
    c = case
    if c["op"] == "swiglu":
        # four-bit values of computed numbers: one on a rounding boundary may go either way, and
        # the last bit of a sum decides it
        return None
    s = prepare(case, seed)
    if c["op"] == "quant":
        return _e2m1_64(s["x"].double())
    if c["op"] == "norm":
        r, x = _norm_64(s)
        return {"residual": r, "x": x}
    if c["op"] == "gemm":
        off = s["offsets"].tolist()
        a = _mx4_64(s["a"], s["a_s"])
        out = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device="cuda")
        for g in range(c["groups"]):
            lo, hi = off[g], off[g + 1]
            if lo == hi:
                continue
            out[lo:hi] = a[lo:hi] @ _mx4_64(s["w"][g], s["w_s"][g]).t()
        return out
    # the layer: routing in fp64, then expert by expert over the tokens that chose it
    E, S = c["experts"], c["shared"]
    x = s["x"].double()
    bias = None if s["e_bias"] is None else s["e_bias"].double()
    logits = x @ s["wg"].double().t()
    score = 1.0 / (1.0 + torch.exp(-logits)) if c["scoring"] == "sigmoid" else logits
    sel = (score if bias is None else score + bias).cpu().numpy()
    score, logits = score.cpu().numpy(), logits.cpu().numpy()
    weight = np.zeros((c["tokens"], E + S))
    weight[:, E:] = 1.0
    per = E // c["num_groups"]
    for t in range(c["tokens"]):
        best = sorted(range(c["num_groups"]), key=lambda g: (-np.sort(
            sel[t, g * per:(g + 1) * per])[::-1][:c["group_topn"]].sum(), g))
        kept = set(best[:c["topk_groups"]])
        ids = sorted((e for e in range(E) if e // per in kept), key=lambda e: (-sel[t, e], e))
        ids = ids[:c["top_k"]]
        z = score[t] if c["scoring"] == "sigmoid" else np.exp(logits[t] - logits[t].max())
        total = z[ids].sum() if c["norm"] else (z.sum() if c["scoring"] == "softmax" else 1.0)
        weight[t, ids] = z[ids] / total * c["scaling"]
    chosen = weight != 0
    rounded = {"bf16": lambda v: v, "fp8": _e4m3_64, "mxfp4": _e2m1_64}[c["dtype"]]
    xq = rounded(x)
    out = torch.zeros_like(x)
    for e in range(E + S):
        rows = np.nonzero(chosen[:, e])[0]
        if not len(rows):
            continue
        if c["dtype"] == "bf16":
            w13, w2 = s["w13"][e].double(), s["w2"][e].double()
        elif c["dtype"] == "fp8":
            up = lambda t: t.double().repeat_interleave(128, 0).repeat_interleave(128, 1)  # noqa: E731
            w13 = s["w13"][e].double() * up(s["w13_s"][e])
            w2 = s["w2"][e].double() * up(s["w2_s"][e])
        else:
            w13, w2 = _mx4_64(s["w13"][e], s["w13_s"][e]), _mx4_64(s["w2"][e], s["w2_s"][e])
        rows = torch.tensor(rows, device="cuda")
        o = xq[rows] @ w13.t()
        h = rounded(_silu64(o[:, :c["inter"]]) * o[:, c["inter"]:])
        p = torch.tensor(weight[:, e], device="cuda")[rows, None]
        out[rows] += p * (h @ w2.t())
    return out


def _norm_64(s):
    c = s["case"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    H = c["hidden"]

    def unit(v, key):
        mean = v.sum(-1, keepdim=True) / H if c["kind"] == "layer" else 0.0
        var = ((v - mean) ** 2).sum(-1, keepdim=True) / H
        out = (v - mean) / torch.sqrt(var + 1e-6) * d["w_" + key]
        return out + d["b_" + key] if "b_" + key in d else out

    n = unit(d["y"], "post") if c["post"] else d["y"]
    if "gate" in d:
        n = n * (d["gate"][:, None] if c["gate"] == "token" else d["gate"])
    r = d["res"] * c["alpha"] + n * c["beta"]
    return r, unit(r, "pre") if c["pre"] else None
