"""Two MoE blocks of a decoder, each x = norm(r), y = MoE(x), r = r + gate * norm(y), over a prompt
and then token by token, with the experts in MXFP4.

  python examples/moe_block.py [--hidden 2048] [--experts 64] [--prompt 300] [--steps 4]

Random weights; prints the time of the prompt and of a decode step, and how far the prompt's path
and the few-token path are apart on the same tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import moe_expert_layer_07_gb300 as moe  # noqa: E402
import synth  # noqa: E402


def make_blocks(shape, count, max_tokens, seed=0):
    blocks = []
    for i in range(count):
        w = synth.make_inputs(shape, seed=seed + i, device="cuda")
        for key in ("w13", "w2"):   # bf16 experts to four bits
            w[key], w[key + "_s"] = moe.mx4_quantize(w[key])
        import dataclasses
        layer = moe.Mx4MoELayer(dataclasses.replace(shape, dtype="mxfp4"), w, max_tokens)
        ones = torch.ones(shape.hidden, dtype=torch.bfloat16, device="cuda")
        gate = torch.full_like(ones, 0.5)
        blocks.append(moe.MoEBlock(layer, ones, w_post=ones, gate=gate))
    return blocks


def run(blocks, residual):
    """All blocks over the rows of residual, in place: one norm pass between two layers."""
    x = torch.empty(residual.shape, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    blocks[0].pre(residual, x)
    for b, after in zip(blocks, blocks[1:] + [None]):
        b.forward(residual, x, y, w_next=after and after.w_pre, x_next=None if after is None else x)
    return residual


def timed(f):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    f()
    a.record()
    f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    for name, default in (("hidden", 2048), ("inter", 1408), ("experts", 64), ("top-k", 6),
                          ("prompt", 300), ("steps", 4)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    shape = synth.MoEShape("example", tokens=a.prompt, hidden=a.hidden, inter=a.inter,
                           num_experts=a.experts, num_shared=1, top_k=a.top_k)
    blocks = make_blocks(shape, 2, a.prompt)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randn(a.prompt, a.hidden, device="cuda", generator=g)
    out = run(blocks, prompt.clone())
    print(f"prompt of {a.prompt}: {timed(lambda: run(blocks, prompt.clone())):.3f} ms")
    for step in range(a.steps):
        few = run(blocks, prompt[step:step + 1].clone())
        off = float((few - out[step:step + 1]).abs().max() / out[step].abs().max())
        print(f"token {step}: alone against in the prompt, largest difference {off:.1e} of the largest value")
    one = prompt[:1].clone()
    print(f"decode step: {1e3 * timed(lambda: run(blocks, one)):.1f} us")
    if any(b.layer.status() for b in blocks):
        raise SystemExit("a device status bit is set")


if __name__ == "__main__":
    main()
