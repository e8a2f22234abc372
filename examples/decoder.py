"""Layers of a decoder, attention over a cache in four bits and then experts in four bits, over a batch
of prompts and then token by token, the decode step as a CUDA graph.

  python examples/decoder.py [--hidden 1024] [--layers 2] [--requests 3] [--prompt 100] [--steps 8]

Random weights; the "next token" of a request is its last residual row, scaled.  Prints the time of the
prompts and of a decode step, and how far a step's rows are from those of one long prompt."""
import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import moe_expert_layer_07_gb300 as moe  # noqa: E402
import synth  # noqa: E402


class Decoder:
    """Layers that share one PageTables; each has a cache of its own with the same page numbers."""

    def __init__(self, hidden, layers, requests, max_len, max_rows, q_heads=8, kv_heads=2, dim=128, page=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        shape = synth.MoEShape("decoder", tokens=max_rows, hidden=hidden, inter=hidden // 2, num_experts=16,
                               num_shared=1, top_k=4)
        four = dataclasses.replace(shape, dtype="mxfp4")
        max_pages = -(-max_len // page)
        pages = requests * max_pages
        ones, gate = torch.ones(hidden, **bf16), torch.full((hidden,), 0.5, **bf16)
        table = moe.rope_table(max_len, dim)
        self.layers = []

        def weights(n, k):
            return moe.mx4_quantize((torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).bfloat16())
        for i in range(layers):
            cache = moe.Cache4(pages, page, kv_heads, dim)
            head = 1 + 0.1 * torch.randn(2, dim, device="cuda", generator=g)
            attention = moe.AttentionBlock(
                cache, q_heads, hidden, weights((q_heads + 2 * kv_heads) * dim, hidden), weights(hidden, q_heads * dim),
                table, requests, max_rows, max_pages, max_q=max_len, max_len=max_len, w_q=head[0].bfloat16(),
                w_k=head[1].bfloat16(), w_pre=ones, w_post=ones, gate=gate)
            w = synth.make_inputs(shape, seed=seed + i, device="cuda")
            for key in ("w13", "w2"):
                w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
            self.layers.append((attention, moe.MoEBlock(moe.Mx4MoELayer(four, w, max_rows), ones, w_post=ones, gate=gate)))
        self.tables = moe.PageTables(self.layers[0][0].cache, requests, max_pages, max_rows)
        self.x, self.y = torch.empty(max_rows, hidden, **bf16), torch.empty(max_rows, hidden, **bf16)

    def forward(self, residual, new_tokens):
        """Rows of new tokens, request after request, through all layers, in place."""
        T = residual.shape[0]
        x, y = self.x[:T], self.y[:T]
        self.tables.step(new_tokens)
        self.layers[0][0].pre(residual, x)
        for i, (attention, experts) in enumerate(self.layers):
            attention.forward(residual, x, y, self.tables, w_next=experts.w_pre, x_next=x)
            after = self.layers[i + 1][0].w_pre if i + 1 < len(self.layers) else None
            experts.forward(residual, x, y, w_next=after, x_next=None if after is None else x)
        return residual

    def status(self):
        bits = int(self.tables.status)
        for attention, experts in self.layers:
            bits |= attention.status() | experts.layer.status()
        return bits


def timed(f):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    for name, default in (("hidden", 1024), ("layers", 2), ("requests", 3), ("prompt", 100), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    R, total = a.requests, a.prompt + a.steps
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(R, total, a.hidden, device="cuda", generator=g)
    counts = lambda n: torch.full((R,), n, dtype=torch.int32, device="cuda")  # noqa: E731
    one = Decoder(a.hidden, a.layers, R, total, R * total)
    long = one.forward(rows.reshape(R * total, -1).clone(), counts(total)).reshape(R, total, -1)
    model = Decoder(a.hidden, a.layers, R, total, R * max(a.prompt, 1))
    prompt = rows[:, :a.prompt].reshape(R * a.prompt, -1).clone()
    print(f"{R} prompts of {a.prompt}: {timed(lambda: model.forward(prompt, counts(a.prompt))):.3f} ms")
    step, ones = torch.empty(R, a.hidden, device="cuda"), counts(1)
    saved = [t.clone() for t in (model.tables.lengths, model.tables.table, model.tables.free_range)]
    step.copy_(rows[:, a.prompt])
    model.forward(step, ones)   # once outside the graph, then back to where it was
    for t, s in zip((model.tables.lengths, model.tables.table, model.tables.free_range), saved):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model.forward(step, ones)
    for i in range(a.steps):
        step.copy_(rows[:, a.prompt + i])
        ms = timed(graph.replay)
        want = long[:, a.prompt + i]
        off = float((step - want).norm() / want.norm())
        print(f"step {i}: {1e3 * ms:.1f} us, {off:.3f} from the long prompt's rows")
    if model.status() or one.status():
        raise SystemExit("a device status bit is set")


if __name__ == "__main__":
    main()
