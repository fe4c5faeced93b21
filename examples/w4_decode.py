"""Greedy decoding with 4-bit weights: the operators together, as a server would use them.

    python examples/w4_decode.py [--tokens T] [--steps N] [--layers L] [--hidden H]
                                 [--inter I] [--experts E] [--topk K] [--vocab V] [--group G]

A stack of MoE layers (no attention, which is not this library's) between an embedding
and an output projection, with random weights.  Each layer's router and the output
projection are moe_w4_matvec with fp32 results, its experts moe_w4_forward; a step of T
sequences is one CUDA graph.  The first step's logits are checked against a plain fp32
form of it on the GPU, which takes the same experts: a pair of nearly equal router
logits may fall either way.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_layer_align_gb300 as moe  # noqa: E402


def quantize(w, group):
    """[.., N, K] to codes, scales and zero points, group by group: the range of the
    group's values (and 0) in 15 steps."""
    K = w.shape[-1]
    pad = -K % group
    g = torch.nn.functional.pad(w, (0, pad)).unflatten(-1, (-1, group))
    lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    scale = ((hi - lo) / 15).clamp(min=1e-8).to(torch.bfloat16)
    zero = (-lo / scale.float()).round().clamp(0, 15)
    q = (g / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15)
    q = q.flatten(-2)[..., :K].to(torch.uint8)
    codes = (q[..., 0::2] | q[..., 1::2] << 4).contiguous()
    return moe.W4Tensor(codes, scale.contiguous(), zero.to(torch.uint8).contiguous(), group=group)


def plain(w: moe.W4Tensor):
    """The fp32 values of a weight."""
    K = w.shape[-1]
    q = torch.stack((w.codes & 15, w.codes >> 4), -1).flatten(-2).float()

    def spread(t):
        return t.float().repeat_interleave(w.group, -1)[..., :K]

    return (q - spread(w.zeros)) * spread(w.scales)


def norm(x):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Model:
    def __init__(self, layers, hidden, inter, experts, topk, vocab, group, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5
            return quantize(w, group)

        self.sizes = dict(H=hidden, I=inter, E=experts, top_k=topk)
        self.topk = topk
        self.embedding = torch.randn(vocab, hidden, generator=g, device="cuda")
        self.layers = [dict(router=weight(experts, hidden), w13=weight(experts, 2 * inter, hidden),
                            w2=weight(experts, hidden, inter)) for _ in range(layers)]
        self.head = weight(vocab, hidden)

    def plan(self, T):
        """The buffers that a server keeps for T sequences."""
        s, V = self.sizes, self.head.shape[0]

        def scratch(K):
            n = moe.moe_w4_matvec_scratch_size(T, K)
            return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None

        return dict(workspace=moe.alloc_w4_workspace(T, s["H"], s["I"], s["E"], s["top_k"]),
                    scratch=scratch(s["H"]),
                    router=torch.empty(T, s["E"], device="cuda"),
                    y=torch.empty(T, s["H"], dtype=torch.bfloat16, device="cuda"),
                    logits=torch.empty(T, V, device="cuda"))

    def step(self, ids, plan, experts=None):
        """Logits of the tokens that follow `ids` [T].  `experts`: a list that gets the
        layers' choices [T, top_k]."""
        x = self.embedding[ids]
        for layer in self.layers:
            h = norm(x).to(torch.bfloat16)
            moe.moe_w4_matvec(h, layer["router"], out=plan["router"], scratch=plan["scratch"])
            if experts is not None:
                experts.append(torch.empty(len(ids), self.topk, dtype=torch.int32, device="cuda"))
            moe.moe_w4_forward(h, plan["router"], layer["w13"], layer["w2"], self.topk,
                               out=plan["y"], workspace=plan["workspace"],
                               topk_ids_out=experts[-1] if experts else None)
            x = x + plan["y"].float()
        return moe.moe_w4_matvec(norm(x).to(torch.bfloat16), self.head, out=plan["logits"],
                                 scratch=plan["scratch"])

    def plain_step(self, ids, experts):
        """step in plain fp32, with the experts that it took; and by how much of a
        probability a better expert was passed over."""
        x, missed = self.embedding[ids], 0.0
        I = self.sizes["I"]
        for layer, which in zip(self.layers, experts):
            h = norm(x).to(torch.bfloat16).float()
            p = torch.softmax(h @ plain(layer["router"]).T, -1)
            w = p.gather(1, which.long())
            rest = p.scatter(1, which.long(), 0.0)
            missed = max(missed, (rest.amax(-1) / w.amin(-1) - 1).max().item())
            w = w / w.sum(-1, keepdim=True)
            y = torch.zeros_like(x)
            for e in which.unique().tolist():
                t, slot = (which == e).nonzero(as_tuple=True)
                gu = h[t] @ plain(moe.W4Tensor(*(v[e] for v in (
                    layer["w13"].codes, layer["w13"].scales, layer["w13"].zeros)),
                    group=layer["w13"].group)).T
                a = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
                d = a @ plain(moe.W4Tensor(*(v[e] for v in (
                    layer["w2"].codes, layer["w2"].scales, layer["w2"].zeros)),
                    group=layer["w2"].group)).T
                y.index_add_(0, t, w[t, slot, None] * d)
            x = x + y.to(torch.bfloat16).float()
        return norm(x).to(torch.bfloat16).float() @ plain(self.head).T, missed


def decode(model, T, steps):
    """`steps` greedy tokens of T sequences; returns (tokens [steps, T], us a step)."""
    plan = model.plan(T)
    ids = torch.arange(T, device="cuda") % model.head.shape[0]
    start = ids.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.step(ids, plan)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids.copy_(model.step(ids, plan).argmax(-1))
    ids.copy_(start)
    tokens = torch.empty(steps, T, dtype=torch.long, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for i in range(steps):
        graph.replay()
        tokens[i].copy_(ids)
    b.record()
    b.synchronize()
    status = moe.moe_check_status(plan["workspace"])
    if status:
        raise moe.MoeError(status, "moe_w4_forward")
    return tokens, a.elapsed_time(b) * 1e3 / steps


def main(argv=None):
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 1), ("steps", 64), ("layers", 4), ("hidden", 2048),
                        ("inter", 768), ("experts", 128), ("topk", 8), ("vocab", 32768),
                        ("group", 128)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args(argv)
    torch.backends.cuda.matmul.allow_tf32 = False
    model = Model(a.layers, a.hidden, a.inter, a.experts, a.topk, a.vocab, a.group)
    ids = torch.arange(a.tokens, device="cuda") % a.vocab
    experts = []
    got = model.step(ids, model.plan(a.tokens), experts)
    want, missed = model.plain_step(ids, experts)
    off = ((got - want).norm() / want.norm()).item()
    tokens, us = decode(model, a.tokens, a.steps)
    print(f"{a.tokens} sequences, {a.layers} layers: {us:.1f} us a step, "
          f"{a.tokens / us * 1e6:.0f} tokens/s; logits off by {off:.1e} of their norm, "
          f"experts passed over by {max(missed, 0):.1e} of their probability; "
          f"first tokens {tokens[:8, 0].tolist()}")
    return off, missed, tokens


if __name__ == "__main__":
    main()
