"""A decoder layer built from the library's operators, used as a program uses
them: a prompt through the chunked forward, then single tokens on the same
pool slots, then one training step's gradients.

    python examples/linear_attention_block.py [--layers 2] [--prompt 300] [--tokens 8]

Layer (D = nv * V channels): x -> norm -> projection -> causal Conv1d with SiLU
-> linear attention with a decay for each head -> norm per head, gated ->
projection -> norm, gate and residual scale, fused with the next layer's norm.
Projections are torch matrix products with random weights.  The program checks
that token-by-token decoding continues the prompt: the last tokens' outputs
agree with those of one forward over the whole sequence.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_loop_amd as gdr  # noqa: E402

NK, NV, K, V = 4, 8, 64, 64
D = NV * V
CONV = 2 * NK * K + NV * V


class Layer:
    """Weights, pool slots and the operators of one layer."""

    def __init__(self, gen, slots, dtype):
        def normal(*shape, std):
            return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

        self.w_qkv = normal(D, CONV, std=D ** -0.5)
        self.w_gate = normal(D, D, std=D ** -0.5)
        self.w_decay = normal(D, NV, std=D ** -0.5)
        self.w_out = normal(D, D, std=D ** -0.5)
        self.conv = torch.randn((CONV, 4), generator=gen, device="cuda") * 0.5
        self.head_norm = torch.ones(V, device="cuda")       # shared by the heads
        self.post_norm = torch.ones(D, device="cuda")
        self.pre_norm = torch.ones(D, device="cuda")        # of the next layer
        self.channel_gate = torch.full((D,), 0.5, device="cuda")
        self.conv_state = torch.zeros((slots, 3, CONV), device="cuda", dtype=dtype)
        self.state = torch.zeros((slots, NV, K, V), device="cuda")

    def project(self, n, offsets, slots):
        qkv = gdr.gdr_causal_conv1d(n @ self.w_qkv, self.conv, offsets, silu=True,
                                    conv_state=self.conv_state, slot_idx=slots)
        q = qkv[:, :NK * K].unflatten(1, (NK, K))
        k = qkv[:, NK * K:2 * NK * K].unflatten(1, (NK, K))
        v = qkv[:, 2 * NK * K:].unflatten(1, (NV, V))
        g = -torch.nn.functional.softplus(n @ self.w_decay)
        return q, k, v, g, n @ self.w_gate

    def finish(self, o, gate, x):
        """Gated norm per head, output projection, and the norms around the residual."""
        h, _ = gdr.gdr_block_norm(o.flatten(1), post_weight=self.head_norm, group=V, gate=gate,
                                  activation="silu")
        return gdr.gdr_block_norm(h @ self.w_out, post_weight=self.post_norm,
                                  gate=self.channel_gate, residual=x, residual_scale=0.7,
                                  pre_weight=self.pre_norm)

    def prompt(self, x, n, offsets, slots):
        q, k, v, g, gate = self.project(n, offsets, slots)
        o, _ = gdr.gdr_linear_attention_fwd(q, k, v, g, offsets, state=self.state, slot_idx=slots)
        return self.finish(o, gate, x)

    def step(self, x, n, offsets, slots):
        q, k, v, g, gate = self.project(n, offsets, slots)
        o = gdr.gdr_linear_attention_step(q, k, v, g, self.state, slots)
        return self.finish(o, gate, x)


def offsets_of(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def generate(layers, x, lens, slots, tokens):
    """The prompts' rows of x, then `tokens` single tokens a row; x [rows][len + tokens, D]."""
    def through(rows, form):
        offs = offsets_of([r.shape[0] for r in rows])
        x = torch.cat(rows)
        _, n = gdr.gdr_block_norm(x, pre_weight=layers[0].pre_norm)
        for layer in layers:
            x, n = getattr(layer, form)(x, n, offs, slots)
        return n

    out = [list(through([r[:m] for r, m in zip(x, lens)], "prompt").split(lens))]
    for t in range(tokens):
        out.append(list(through([r[m + t:m + t + 1] for r, m in zip(x, lens)], "step").split(1)))
    return [torch.cat([o[r] for o in out]) for r in range(len(lens))]


def train_step(layer, x, lens):
    """Gradients of a layer's attention and norms for a loss of sum(h * target)."""
    offs = offsets_of(lens)
    q = torch.randn((x.shape[0], NK, K), device="cuda", dtype=x.dtype) * K ** -0.25
    k, v = torch.randn_like(q) * K ** -0.25, torch.randn((x.shape[0], NV, V), device="cuda",
                                                         dtype=x.dtype)
    g = -torch.nn.functional.softplus(torch.randn((x.shape[0], NV), device="cuda") - 2)
    gate, target = torch.randn_like(x), torch.randn_like(x)
    o, _ = gdr.gdr_linear_attention_fwd(q, k, v, g, offs)
    args = dict(post_weight=layer.head_norm, group=V, gate=gate, activation="silu")
    h, _ = gdr.gdr_block_norm(o.flatten(1), residual=x, **args)
    dx, dgate, do, dw, _ = gdr.gdr_block_norm_bwd(target, None, o.flatten(1), None, **args)
    grads = gdr.gdr_linear_attention_bwd(do.unflatten(1, (NV, V)), q, k, v, g, offs)
    return h, (dx, dgate, dw) + tuple(t for t in grads if t is not None)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    lens = [a.prompt, max(1, a.prompt // 3), 1]
    rows = [torch.randn((n + a.tokens, D), generator=gen, device="cuda") for n in lens]
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")

    def fresh():
        g = torch.Generator(device="cuda").manual_seed(1)
        return [Layer(g, 4, torch.float32) for _ in range(a.layers)]

    with torch.no_grad():
        parts = generate(fresh(), rows, lens, slots, a.tokens)
        whole = generate(fresh(), rows, [n + a.tokens for n in lens], slots, 0)
        worst = max(float((p - w).abs().max() / w.abs().max()) for p, w in zip(parts, whole))
        print(f"{a.layers} layers, prompts of {lens} tokens and {a.tokens} more: "
              f"step by step against one forward {worst:.1e}")
        h, grads = train_step(fresh()[0], rows[0], [rows[0].shape[0]])
        print("training step:", ", ".join(f"{tuple(t.shape)}" for t in grads))
    finite = all(torch.isfinite(t).all() for t in (h, *grads))
    return worst, finite


if __name__ == "__main__":
    worst, finite = main()
    if worst > 1e-4 or not finite:
        sys.exit(1)
