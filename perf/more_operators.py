"""What is measured of the operators of attention over a cache in four bits: the tables of its
pages, the norm and rotation of queries and keys with the cache's write, the attention itself, and
products of a few rows with four-bit weights.

Each case names one operator and its sizes.  ``run`` computes it either in plain fp32 torch
operations or, with ``own`` set, by the library's entry points; ``exact`` computes it in fp64.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32          # elements that share one MXFP4 scale

# ---- cases ---------------------------------------------------------------------------


def listed():
    return [
        # a small server's decode step: one token more for each of eight requests
        dict(name="tables_step_b8", op="tables", requests=8, page=64, held=8192, new=1, mix=1),
        # a large step that mixes requests which decode with prompts that have just arrived
        dict(name="tables_mixed_b1000", op="tables", requests=1000, page=16, held=4096, new=96, mix=2),
        # the norm and rotation of one decode step of seven requests, into the cache
        dict(name="rope_step_t7", op="rope", tokens=7, q_heads=64, kv_heads=8, dim=128, rot=128,
             style="halves", norm=True, cache=True, page=64, far=8192),
        # a long prompt, q and k kept in bf16
        dict(name="rope_prompt_t8192", op="rope", tokens=8192, q_heads=64, kv_heads=8, dim=128, rot=128,
             style="halves", norm=True, cache=False, page=64, far=8192),
        # a prompt into the cache: narrow heads, half of each rotated, neighbours in pairs
        dict(name="rope_store_t5001", op="rope", tokens=5001, q_heads=32, kv_heads=4, dim=64, rot=32,
             style="pairs", norm=True, cache=True, page=16, far=131072),
        # one user's next token: a cache of a few megabytes, latency is most of it
        dict(name="attn_step_b1", op="attn", requests=1, q_heads=64, kv_heads=8, dim=128, page=64,
             shortest=4097, longest=4097, fewest=1, most=1, window=0, lse=False, mix=3),
        # a server's decode step: 48 requests of very different lengths
        dict(name="attn_step_b48", op="attn", requests=48, q_heads=64, kv_heads=8, dim=128, page=64,
             shortest=64, longest=16384, fewest=1, most=1, window=0, lse=False, mix=4),
        # two very long documents, five query heads to a key head, three drafted tokens each
        dict(name="attn_long_b2", op="attn", requests=2, q_heads=40, kv_heads=8, dim=128, page=16,
             shortest=131073, longest=131073, fewest=3, most=3, window=0, lse=True, mix=5),
        # chunks of prompts onto what is in the cache already: the tensor cores' work
        dict(name="attn_prompt_b3", op="attn", requests=3, q_heads=64, kv_heads=8, dim=128, page=32,
             shortest=1500, longest=8192, fewest=500, most=4096, window=0, lse=False, mix=6),
        # queries, keys and values of one token from MXFP4 weights
        dict(name="w4_mx_t1", op="w4", rows=1, n=10240, k=7168, kind="mx", group=32, zeros=False,
             out="bf16"),
        # the product behind attention for sixteen requests, four-bit integers with zero points
        dict(name="w4_int_t16", op="w4", rows=16, n=7168, k=8192, kind="int", group=128, zeros=True,
             out="bf16"),
        # a small layer with an odd number of outputs, three rows
        dict(name="w4_mx_t3_small", op="w4", rows=3, n=1111, k=1024, kind="mx", group=32, zeros=False,
             out="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "attn", "attn", "attn", "w4", "w4"])
    mix = rng.randrange(1 << 30)
    if op == "tables":
        return dict(op="tables", requests=_log_int(rng, 1, 1000), page=rng.choice([16, 32, 64, 128]),
                    held=_log_int(rng, 1, 16384), new=_log_int(rng, 1, 96), mix=mix)
    if op == "rope":
        dim = rng.choice([64, 128])
        kv = _log_int(rng, 1, 8)
        return dict(op="rope", tokens=_log_int(rng, 1, 8192), q_heads=kv * rng.randint(1, 8), kv_heads=kv,
                    dim=dim, rot=rng.choice([dim, dim, dim // 2]), style=rng.choice(["halves", "pairs"]),
                    norm=rng.random() < 0.7, cache=rng.random() < 0.5, page=rng.choice([16, 64]),
                    far=_log_int(rng, 256, 131072))
    if op == "attn":
        kv, dim = _log_int(rng, 1, 8), rng.choice([64, 128, 128])
        c = dict(op="attn", q_heads=kv * rng.randint(1, 8), kv_heads=kv, dim=dim,
                 page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, _log_int(rng, 1, 4096)]),
                 lse=rng.random() < 0.3, mix=mix)
        if rng.random() < 0.6:   # decode, with drafted tokens now and then
            requests = _log_int(rng, 1, 48)
            longest = _log_int(rng, 1, min(131072, 262144 // requests))
            c.update(requests=requests, shortest=_log_int(rng, 1, longest), longest=longest,
                     fewest=1, most=rng.choice([1, 1, 2, 5]))
        else:                    # chunks of prompts
            requests = _log_int(rng, 1, 4)
            longest = _log_int(rng, 32, 8192)
            most = _log_int(rng, 16, 4096 // requests)
            c.update(requests=requests, shortest=_log_int(rng, 16, longest), longest=longest,
                     fewest=_log_int(rng, 1, most), most=most)
        return c
    kind = rng.choice(["mx", "int"])
    group = 32 if kind == "mx" else rng.choice([32, 64, 128])
    return dict(op="w4", rows=_log_int(rng, 1, 16), n=_log_int(rng, 16, 10240), k=group * _log_int(rng, 1, 8192 // group),
                kind=kind, group=group, zeros=kind == "int" and rng.random() < 0.5,
                out=rng.choice(["bf16", "bf16", "fp32"]))


# ---- lengths: from the case alone ---------------------------------------------------------


def _spread(g, lo, hi, n):
    """n whole numbers from lo to hi, spread over their logarithm, the largest among them."""
    v = np.exp(g.uniform(math.log(lo), math.log(hi), n)) if hi > lo else np.full(n, float(lo))
    v = np.clip(np.rint(v), lo, hi).astype(np.int64)
    v[g.integers(n)] = hi
    return v


def _table_lengths(c):
    """(held, new): two thirds of the requests decode, one in ten waits, the rest are prompts."""
    g = np.random.default_rng(c["mix"])
    held, new = _spread(g, 1, c["held"], c["requests"]), np.ones(c["requests"], np.int64)
    if c["new"] > 1:
        kind = g.random(c["requests"])
        prompt = kind < 0.25
        new[prompt] = _spread(g, 1, c["new"], c["requests"])[prompt]
        held[kind < 0.12] = 0
        new[kind > 0.9] = 0
    return held, new


def _attn_lengths(c):
    """(length with the query tokens, query tokens) of each request."""
    g = np.random.default_rng(c["mix"])
    total = _spread(g, c["shortest"], c["longest"], c["requests"])
    new = _spread(g, c["fewest"], c["most"], c["requests"])
    return np.maximum(total, new), new


def _visible(c):
    """(keys that a request's queries see in all, pairs of a query and a key) of each request."""
    total, new = _attn_lengths(c)
    w = c["window"]
    keys, pairs = [], []
    for L, n in zip(total.tolist(), new.tolist()):
        first = L - n   # position of the first query token
        lo = max(0, first - w + 1) if w else 0
        keys.append(L - lo)
        p = np.arange(first, L, dtype=np.float64) + 1
        pairs.append(float((np.minimum(p, w) if w else p).sum()))
    return keys, pairs


# ---- MXFP4 in plain operations -------------------------------------------------------------

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


# ---- inputs ------------------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    v = torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)
    return (v * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(total, page, seed):
    """(table [requests, most pages], pages): each request's pages, anywhere in the cache."""
    need = -(-total // page)
    order = np.random.default_rng(seed).permutation(int(need.sum()) + 5)
    table = np.zeros((len(total), int(need.max())), np.int64)
    at = 0
    for b, n in enumerate(need.tolist()):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if own:
        import moe_expert_layer_07_gb300 as moe
        s["moe"] = moe
    if c["op"] == "tables":
        held, new = _table_lengths(c)
        g = np.random.default_rng(seed)
        shift = g.permutation(len(held))   # the same requests in another order
        held, new = held[shift], new[shift]
        had = -(-held // c["page"])
        total = -(-(held + new) // c["page"])
        order = g.permutation(int(total.sum()) + 100)
        s["width"] = int(total.max()) + 3
        table = np.full((len(held), s["width"]), -1, np.int64)
        at = 0
        for b, n in enumerate(had.tolist()):
            table[b, :n] = order[at:at + n]
            at += n
        free = order[at:]   # a ring: what is free starts anywhere in it
        turn = int(g.integers(len(free)))
        s.update(held=_i32(held), new=_i32(new), table=_i32(table), free=_i32(np.roll(free, turn)),
                 free_range=torch.tensor([turn, turn + len(free)], dtype=torch.int64, device="cuda"),
                 tokens=int(new.sum()) + 7)   # a step's buffers are as large as the largest step
        if own:
            e = lambda n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
            s.update(lengths=e(len(held)), starts=e(len(held) + 1), slots=e(s["tokens"]),
                     positions=e(s["tokens"]), free_out=e(2, torch.int64))
    elif c["op"] == "rope":
        T, Hq, Hk, D = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
        g = np.random.default_rng(seed)
        s["qkv"] = _randn(gen, T, (Hq + 2 * Hk) * D, dtype=torch.bfloat16, scale=2.0)
        s["pos"] = _i32((int(g.integers(max(1, c["far"] - T + 1))) + np.arange(T)) % c["far"])
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        ang = torch.arange(c["far"], dtype=torch.float64, device="cuda")[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["w_q"] = (1 + _randn(gen, D, scale=0.1)).bfloat16() if c["norm"] else None
        s["w_k"] = (1 + _randn(gen, D, scale=0.1)).bfloat16() if c["norm"] else None
        if own:
            bf = dict(dtype=torch.bfloat16, device="cuda")
            s["q"] = torch.empty(T, Hq, D, **bf)
            s["k"], s["v"] = torch.empty(T, Hk, D, **bf), torch.empty(T, Hk, D, **bf)
        if c["cache"]:
            page = c["page"]
            pages = -(-T // page) + 3
            order = g.permutation(pages)
            at = np.arange(T) + int(g.integers(page))
            s["slots"] = _i32(order[at // page] * page + at % page)
            if own:
                s["cache"] = s["moe"].Cache4(pages, page, Hk, D, device="cuda")
    elif c["op"] == "attn":
        Hq, Hk, D, page = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        total, new = _attn_lengths(c)
        table, pages = _pages(total, page, seed)
        s["q"] = _randn(gen, int(new.sum()), Hq, D, dtype=torch.bfloat16)
        s["codes"] = torch.empty(pages, 2, Hk, page, D // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(pages, 2, Hk, page, D // BLOCK, dtype=torch.uint8, device="cuda")
        # keys have channels that stand out in every token, values heads of different sizes
        lean = _randn(gen, 2, Hk, 1, D) * (torch.rand(2, Hk, 1, D, generator=gen, device="cuda") < 0.05)
        lean[1] = 0
        size = torch.ones(2, Hk, 1, 1, device="cuda")
        size[1] = torch.exp(_randn(gen, Hk, 1, 1, scale=0.5))
        step = max(1, (1 << 26) // (2 * Hk * page * D))   # pages at a time
        for p in range(0, pages, step):
            n = min(step, pages - p)
            v = (_randn(gen, n, 2, Hk, page, D) + 3 * lean) * size
            s["codes"][p:p + n], s["scales"][p:p + n] = _mx4_pack(v.bfloat16().float())
        starts = np.concatenate([[0], np.cumsum(new)])
        s.update(table=_i32(table), lengths=_i32(total), starts=_i32(starts), scale=D ** -0.5,
                 host=(total.tolist(), new.tolist(), starts.tolist()))
        if own:
            s["cache"] = s["moe"].Cache4.of(s["codes"], s["scales"])
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], device="cuda") if c["lse"] else None
            s["plan"] = s["moe"].CacheAttention(c["requests"], s["q"].shape[0], Hq, s["cache"],
                                                table.shape[1], max_q=int(new.max()),
                                                max_len=int(total.max()), window=c["window"],
                                                scale=s["scale"])
    else:
        N, K, G = c["n"], c["k"], c["k"] // c["group"]
        s["x"] = _randn(gen, c["rows"], K, dtype=torch.bfloat16)
        if c["kind"] == "mx":
            s["w"], s["w_s"] = _mx4_pack(_randn(gen, N, K, scale=0.02))
            s["w_z"] = None
        else:
            s["w"] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
            s["w_s"] = (torch.rand(N, G, device="cuda", generator=gen) * 0.004 + 0.002).bfloat16()
            s["w_z"] = torch.randint(6, 11, (N, G), dtype=torch.uint8, device="cuda",
                                     generator=gen) if c["zeros"] else None
        if own:
            s["out"] = torch.empty(c["rows"], N, dtype=_TYPES[c["out"]], device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------


def _plain_tables(s):
    page, held, new, F = s["case"]["page"], s["held"].long(), s["new"].long(), s["free"].shape[0]
    total = held + new
    had, want = (held + page - 1) // page, (total + page - 1) // page
    need = want - had
    zero = held.new_zeros(1)
    page0 = torch.cat([zero, need.cumsum(0)])
    starts = torch.cat([zero, new.cumsum(0)])
    col = torch.arange(s["width"], device=held.device)
    fresh = (col >= had[:, None]) & (col < want[:, None])
    nth = s["free_range"][0] + page0[:-1, None] + col - had[:, None]
    table = torch.where(fresh, s["free"].long()[nth % F], s["table"].long())
    t = torch.arange(s["tokens"], device=held.device)
    b = torch.searchsorted(starts[1:], t, right=True)
    there = b < held.shape[0]
    b = b.clamp(max=held.shape[0] - 1)
    pos = torch.where(there, held[b] + t - starts[b], 0)
    slot = torch.where(there, table[b, pos // page] * page + pos % page, -1)
    i = lambda v: v.to(torch.int32)  # noqa: E731
    return {"table": i(table), "lengths": i(total), "starts": i(starts), "slots": i(slot),
            "positions": i(pos), "free": s["free_range"] + torch.stack([page0[-1], page0[-1] * 0])}


def _turned(c, v, w, cos, sin):
    """v [T, heads, D] normed and rotated, in v's type."""
    if w is not None:
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.to(v.dtype)
    r, h = c["rot"], c["rot"] // 2
    if c["style"] == "halves":
        a, b = v[..., :h], v[..., h:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = v[..., 0:r:2], v[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, v[..., r:]], -1)


def _rope_formula(s, dtype):
    c = s["case"]
    Hq, Hk = c["q_heads"], c["kv_heads"]
    v = s["qkv"].to(dtype).reshape(c["tokens"], -1, c["dim"])
    cs = s["cos_sin"].to(dtype)[s["pos"].long()][:, None]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]
    return (_turned(c, v[:, :Hq], s["w_q"], cos, sin), _turned(c, v[:, Hq:Hq + Hk], s["w_k"], cos, sin),
            v[:, Hq + Hk:])


def _plain_attn(s):
    c = s["case"]
    Hq, Hk, D, page, w = c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["window"]
    out = torch.empty(s["q"].shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    for b, (L, n, at) in enumerate(zip(*s["host"])):
        first = L - n
        lo = max(0, first - w + 1) // page * page if w else 0
        pages = s["table"][b, lo // page:-(-L // page)].long()
        kv = _mx4_values(s["codes"][pages], s["scales"][pages])   # [pages, 2, Hk, page, D]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, Hk, -1, D)[:, :, :L - lo]
        q = s["q"][at:at + n].float().reshape(n, Hk, Hq // Hk, D) * s["scale"]
        key = torch.arange(lo, L, device="cuda")
        row = torch.arange(first, L, device="cuda")[:, None, None]
        hidden = key > row
        if w:
            hidden = hidden | (key <= row - w)
        for h in range(Hk):   # one head at a time: all scores would not fit
            score = torch.matmul(q[:, h], kv[0, h].t()).masked_fill(hidden, -math.inf)
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - top)
            total = p.sum(-1, keepdim=True)
            g = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            out[at:at + n, g] = torch.matmul(p, kv[1, h]) / total
            lse[at:at + n, g] = (top + torch.log(total))[..., 0]
    return {"out": out.bfloat16(), "lse": lse if c["lse"] else None}


def _int_values(s, dtype):
    both = torch.stack([s["w"] & 15, s["w"] >> 4], -1).reshape(s["w"].shape[0], -1, s["case"]["group"])
    zero = 8 if s["w_z"] is None else s["w_z"].to(dtype).unsqueeze(-1)
    return ((both.to(dtype) - zero) * s["w_s"].to(dtype).unsqueeze(-1)).flatten(1)


def run(state):
    s, c = state, state["case"]
    if own:
        moe = s["moe"]
        if c["op"] == "tables":
            moe.cache_tables(s["held"], s["new"], s["free"], s["free_range"], c["page"], s["table"],
                             s["lengths"], s["starts"], s["slots"], s["positions"], s["free_out"])
            return {"table": s["table"], "lengths": s["lengths"], "starts": s["starts"],
                    "slots": s["slots"], "positions": s["positions"], "free": s["free_out"]}
        if c["op"] == "rope":
            style = moe.ROPE_HALVES if c["style"] == "halves" else moe.ROPE_PAIRS
            to = dict(cache=s["cache"], slots=s["slots"]) if c["cache"] else dict(k_out=s["k"])
            moe.qk_norm_rope(s["qkv"], s["pos"], s["cos_sin"], c["q_heads"], c["kv_heads"], s["q"],
                             w_q=s["w_q"], w_k=s["w_k"], eps=1e-6, style=style, **to)
            if c["cache"]:
                moe.cache_read(s["cache"], s["slots"], s["k"], s["v"])
            return {"q": s["q"], "k": s["k"], "v": s["v"] if c["cache"] else None}
        if c["op"] == "attn":
            s["plan"].forward(s["q"], s["table"], s["lengths"], s["starts"], s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        return moe.w4_matvec(s["x"], s["w"], s["w_s"], s["out"], zeros=s["w_z"])
    if c["op"] == "tables":
        return _plain_tables(s)
    if c["op"] == "rope":
        q, k, v = _rope_formula(s, torch.float32)
        if c["cache"]:
            return {"q": q.bfloat16(), "k": _mx4_round(k).bfloat16(), "v": _mx4_round(v).bfloat16()}
        return {"q": q.bfloat16(), "k": k.bfloat16(), "v": None}
    if c["op"] == "attn":
        return _plain_attn(s)
    w = _mx4_values(s["w"], s["w_s"]) if c["kind"] == "mx" else _int_values(s, torch.float32)
    return torch.matmul(s["x"].float(), w.t()).to(_TYPES[c["out"]])


# ---- what a pass cannot do without -----------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "tables":
        held, new = _table_lengths(c)
        fresh = int((-(-(held + new) // c["page"]) - -(-held // c["page"])).sum())
        B, T = len(held), int(new.sum())
        # tokens in a page that a request had: one entry read for each such request
        return {"bytes": 8.0 * B + 8.0 * B + 8.0 * fresh + 8.0 * T + 4.0 * B + 32, "flops": 0.0}
    if c["op"] == "rope":
        T, Hq, Hk, D, R = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["rot"]
        read = 2.0 * (Hq + (2 if c["cache"] else 1) * Hk) * D
        # with a cache: written in four bits and read back from there
        keys = Hk * (4 * (D / 2 + D / BLOCK) + 4 * D) + 8 if c["cache"] else 2 * Hk * D
        return {"bytes": T * (read + 2 * Hq * D + keys + 4) + 4.0 * R * min(T, c["far"]),
                "flops": T * (Hq + Hk) * (5.0 * D + 3 * R)}
    if c["op"] == "attn":
        keys, pairs = _visible(c)
        total, new = _attn_lengths(c)
        D, T = c["dim"], int(new.sum())
        return {"bytes": sum(keys) * c["kv_heads"] * 2 * (D / 2 + D / BLOCK) + 4.0 * T * c["q_heads"] * D
                + (4.0 * T * c["q_heads"] if c["lse"] else 0) + sum(4.0 * (k // c["page"]) for k in keys),
                "flops": 4.0 * D * c["q_heads"] * sum(pairs)}
    T, N, K, G = c["rows"], c["n"], c["k"], c["k"] // c["group"]
    scales = N * G * (1 if c["kind"] == "mx" else 3 if c["zeros"] else 2)
    return {"bytes": N * K / 2 + scales + 2.0 * T * K + (2.0 if c["out"] == "bf16" else 4.0) * T * N,
            "flops": 2.0 * T * N * K}


# ---- the definitions in fp64 ------------------------------------------------------------------


def _e2m1_64(codes, bytes_):
    """Values of MXFP4 codes in fp64, from the format's bits: sign, two of exponent, one of mantissa."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
    scale = torch.exp2(bytes_.double() - 127).repeat_interleave(BLOCK, -1)
    return torch.where(nib >= 8, -mag, mag) * scale


def _nearest_64(v):
    """v fp64 to the nearest value of its block's MXFP4 form, ties to the even code."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(min=-127).double()   # floor(log2(amax)) - 2
    e = torch.where(amax > 0, e, torch.zeros_like(amax))
    a = b.abs() / torch.exp2(e)
    best = torch.zeros_like(a)
    off = a.clone()   # distance from 0
    for i, x in enumerate(_E2M1[1:], 1):
        d = (a - x).abs()
        better = (d < off) | ((d == off) & (i % 2 == 0))
        best, off = torch.where(better, torch.full_like(best, x), best), torch.where(better, d, off)
    return (torch.copysign(best, b) * torch.exp2(e)).reshape(v.shape)


def _exact_attn(s, c):
    total, new, starts = s["host"]
    Hq, Hk, D, page, w = c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["window"]
    G = Hq // Hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(len(total)):
        L, n, at = total[b], new[b], starts[b]
        j = torch.arange(L, device="cuda")
        page_of, inside = s["table"][b].long()[j // page], j % page
        for h in range(Hk):
            k = _e2m1_64(s["codes"][page_of, 0, h, inside], s["scales"][page_of, 0, h, inside])
            v = _e2m1_64(s["codes"][page_of, 1, h, inside], s["scales"][page_of, 1, h, inside])
            for i0 in range(0, n, 512):
                i = torch.arange(i0, min(n, i0 + 512), device="cuda")
                p = (L - n) + i
                q = s["q"][at + i, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,jd->igj", q, k) * s["scale"]
                seen = j[None] <= p[:, None]
                if w:
                    seen &= j[None] > p[:, None] - w
                x = torch.where(seen[:, None], x, -math.inf)
                z = torch.logsumexp(x, -1, keepdim=True)
                lse[at + i, h * G:(h + 1) * G] = z[..., 0]
                out[at + i, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", torch.exp(x - z), v)
    return {"out": out, "lse": lse if c["lse"] else None}


def exact(case, seed):
    c = case
    if c["op"] == "tables":   # whole numbers, one request after the other
        s = prepare(case, seed)
        held, new = s["held"].tolist(), s["new"].tolist()
        table, free, F = s["table"].cpu().numpy().copy(), s["free"].tolist(), s["free"].shape[0]
        at, end = s["free_range"].tolist()
        starts, slots, positions, page = [0], [], [], c["page"]
        for b, (h, n) in enumerate(zip(held, new)):
            for i in range(-(-h // page), -(-(h + n) // page)):
                table[b, i] = free[at % F]
                at += 1
            for p in range(h, h + n):
                slots.append(int(table[b, p // page]) * page + p % page)
                positions.append(p)
            starts.append(starts[-1] + n)
        pad = s["tokens"] - len(slots)
        return {"table": _i32(table), "lengths": _i32(np.add(held, new)), "starts": _i32(starts),
                "slots": _i32(slots + [-1] * pad), "positions": _i32(positions + [0] * pad),
                "free": torch.tensor([at, end], dtype=torch.int64, device="cuda")}
    s = prepare(case, seed)
    if c["op"] == "rope":
        T, D, R, Hq, Hk = c["tokens"], c["dim"], c["rot"], c["q_heads"], c["kv_heads"]
        x = s["qkv"].double().reshape(T, Hq + 2 * Hk, D)
        angle = s["cos_sin"].double()[s["pos"].long()]
        z = torch.complex(angle[:, :R // 2], angle[:, R // 2:])[:, None]   # the rotation as a factor
        got = []
        for part, w in ((x[:, :Hq], s["w_q"]), (x[:, Hq:Hq + Hk], s["w_k"])):
            if w is not None:
                part = part / torch.sqrt(torch.mean(part * part, -1, keepdim=True) + 1e-6) * w.double()
            part = part.clone()
            re, im = ((slice(0, R // 2), slice(R // 2, R)) if c["style"] == "halves"
                      else (slice(0, R, 2), slice(1, R, 2)))
            y = torch.complex(part[..., re].contiguous(), part[..., im].contiguous()) * z
            part[..., re], part[..., im] = y.real, y.imag
            got.append(part)
        if not c["cache"]:
            return {"q": got[0], "k": got[1], "v": None}
        return {"q": got[0], "k": _nearest_64(got[1]), "v": _nearest_64(x[:, Hq + Hk:])}
    if c["op"] == "attn":
        if 4.0 * c["dim"] * c["q_heads"] * sum(_visible(c)[1]) > 4e12:
            return None   # minutes in fp64
        return _exact_attn(s, c)
    if c["kind"] == "mx":
        w = _e2m1_64(s["w"], s["w_s"])
    else:
        code = torch.empty(c["n"], c["k"], dtype=torch.float64, device="cuda")
        code[:, 0::2], code[:, 1::2] = (s["w"] % 16).double(), (s["w"] // 16).double()
        z = torch.full_like(s["w_s"], 8.0).double() if s["w_z"] is None else s["w_z"].double()
        w = (code - z.repeat_interleave(c["group"], 1)) * s["w_s"].double().repeat_interleave(c["group"], 1)
    return torch.einsum("tk,nk->tn", s["x"].double(), w)
