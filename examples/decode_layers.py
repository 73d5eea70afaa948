"""Decode steps of a small MoE model with LoRA adapters, through the public calls alone.

Each layer: norm after the block before it and residual add, router, the adapters' deltas and the
experts (bf16 or 4-bit weights). After the last layer the final norm and a 4-bit output head. The
step is captured in a CUDA graph and replayed on new tokens, as a serving loop would.

    python examples/decode_layers.py --tokens 23 --layers 4 --group 128
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_lora_virtual_gb300 as mol  # noqa: E402


class Layer:
    """Random weights of one layer and its buffers for up to `tokens` tokens."""

    def __init__(self, g, tokens, H, I, E, k, L, r, block_m, group):
        def randn(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        def experts(*shape):
            w = randn(*shape, std=shape[-1] ** -0.5)
            return mol.w4_quantize(w, group) if group else w

        self.E, self.k, self.L, self.scale = E, k, L, 0.5
        self.norm = 1 + randn(H, std=0.1)
        self.router = randn(E, H, std=H ** -0.5)
        self.gate_up, self.down = experts(E, 2 * I, H), experts(E, H, I)
        self.a_gu, self.b_gu = randn(E * L, 2 * r, H, std=H ** -0.5), randn(E * L, 2 * I, r, std=0.1)
        self.a_dn, self.b_dn = randn(E * L, r, I, std=I ** -0.5), randn(E * L, H, r, std=0.1)
        pairs = tokens * k
        self.routing = mol.alloc_routing(pairs, E * L, block_m, "cuda")
        self.align_ws = mol.alloc_workspace(pairs, E * L, block_m, "cuda")
        self.inter_gu = torch.empty(pairs, 2 * r, dtype=torch.float32, device="cuda")
        self.inter_dn = torch.empty(pairs, r, dtype=torch.float32, device="cuda")
        self.delta_gu = torch.empty(pairs, 2 * I, dtype=torch.bfloat16, device="cuda")
        self.delta_dn = torch.empty(pairs, H, dtype=torch.bfloat16, device="cuda")

    def __call__(self, y, residual, lora_ids):
        """The block's output and the residual stream, from those of the block before."""
        residual, x = mol.mol_block_norm(y, residual, self.norm)
        ids, weights = mol.mol_moe_route(x @ self.router.T, self.k)
        mol.mol_lora_forward(x, self.k, ids, lora_ids, self.E, self.L, self.a_gu, self.b_gu, 2,
                             self.scale, self.delta_gu.zero_(), self.routing, self.inter_gu,
                             compute_routing=True, workspace=self.align_ws)
        act = mol.mol_moe_gate_up(x, ids, self.gate_up, delta=self.delta_gu)
        mol.mol_lora_forward(act, 1, None, None, self.E, self.L, self.a_dn, self.b_dn, 1,
                             self.scale, self.delta_dn.zero_(), self.routing, self.inter_dn,
                             compute_routing=False, num_tokens=x.shape[0], topk=self.k)
        return mol.mol_moe_down(act, ids, weights, self.down, delta=self.delta_dn), residual


class Model:
    def __init__(self, tokens=23, layers=2, H=1024, I=256, E=32, k=4, L=4, r=16, vocab=5000,
                 block_m=16, group=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(g, tokens, H, I, E, k, L, r, block_m, group) for _ in range(layers)]
        self.embed = torch.randn(vocab, H, generator=g, device="cuda").to(torch.bfloat16)
        self.norm = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.head = mol.w4_quantize(torch.randn(vocab, H, generator=g, device="cuda") * H ** -0.5)

    def __call__(self, tokens, lora_ids):
        """Logits [T, vocab] of one step: tokens int64 [T], lora_ids int32 [T] (-1: no adapter)."""
        residual = self.embed[tokens]
        y = torch.zeros_like(residual)
        for layer in self.layers:
            y, residual = layer(y, residual, lora_ids)
        _, x = mol.mol_block_norm(y, residual, self.norm)
        return mol.mol_w4_linear(x, self.head)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=23, help="sequences in the batch (up to 64)")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--group", type=int, default=128, choices=(0, 32, 64, 128),
                    help="group of the experts' 4-bit weights, 0 for bf16 experts")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    model = Model(tokens=a.tokens, layers=a.layers, group=a.group)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, 5000, (a.tokens,), generator=g, device="cuda")
    lora_ids = torch.randint(-1, 4, (a.tokens,), generator=g, device="cuda").to(torch.int32)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        model(tokens, lora_ids)  # (allocations and library initialisation, before the capture)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = model(tokens, lora_ids)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(3 + a.steps):
        if step == 3:
            begin.record()
        graph.replay()
        tokens.copy_(logits.argmax(-1))  # greedy: the step's choice is the next step's input
    end.record()
    end.synchronize()
    print(f"{a.tokens} tokens, {a.layers} layers: {begin.elapsed_time(end) / a.steps * 1e3:.0f} us "
          f"a step; last choices {tokens[:4].tolist()}")


if __name__ == "__main__":
    main()
