"""Decode steps of a small MoE model with LoRA adapters, through the public calls alone.

Each layer: norm after the block before it and residual add, router, the adapters' deltas and the
experts (bf16 or 4-bit weights); with --heads its attention half before that: norm, 4-bit projection,
rotary positions and the append to a paged cache, attention over the cache, 4-bit output projection.
After the last layer the final norm and a 4-bit output head. The step is captured in a CUDA graph and
replayed on new tokens, as a serving loop would; with attention a prompt goes through the same layers
first.

    python examples/decode_layers.py --tokens 23 --layers 4 --group 128 --heads 16 --kv-heads 2
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_lora_virtual_gb300 as mol  # noqa: E402


class Batch:
    """Where each sequence's tokens lie and how many there are, for caches of `pages` pages; its tensors
    change in place, so that a captured step follows."""

    def __init__(self, sequences, context, page):
        per = -(-context // page)
        self.page, self.pages = page, sequences * per
        self.table = torch.randperm(self.pages, device="cuda").to(torch.int32).view(sequences, per)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def place(self, counts=None):
        """Makes room for one more token a sequence, or for `counts` more: (positions, slots, where
        each sequence's rows begin or None)."""
        if counts is None:
            at = self.lens.clone()
            self.lens += 1
            of, starts = torch.arange(len(at), device="cuda"), None
        else:
            n = torch.tensor(counts, device="cuda")
            of = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), n, output_size=sum(counts))
            starts = torch.zeros(len(counts) + 1, dtype=torch.int32, device="cuda")
            starts[1:] = n.cumsum(0)
            at = (self.lens[of] + torch.arange(len(of), device="cuda") - starts[of]).to(torch.int32)
            self.lens += n.to(torch.int32)
        slots = self.table[of, (at // self.page).long()] * self.page + at % self.page
        return at, slots.to(torch.int32), starts


class Attention:
    """The attention half of a layer: random weights and the layer's cache."""

    def __init__(self, g, H, heads, kv_heads, D, batch, group=128):
        def randn(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(torch.bfloat16)

        self.heads, self.kv_heads, self.D = heads, kv_heads, D
        self.norm = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.qkv = mol.w4_quantize(randn((heads + 2 * kv_heads) * D, H), group)
        self.out = mol.w4_quantize(randn(H, heads * D), group)
        self.rope = mol.rope_frequencies(D, device="cuda")
        shape = (batch.pages, batch.page, kv_heads, D)
        self.k_cache, self.v_cache = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def __call__(self, y, residual, batch, place):
        positions, slots, starts = place
        residual, x = mol.mol_block_norm(y, residual, self.norm)
        rows = mol.mol_w4_linear(x, self.qkv).view(x.shape[0], -1, self.D)
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = mol.mol_cache_append(k, v, self.k_cache, self.v_cache, slots, positions, self.rope, q=q)
        a = mol.mol_paged_attention(q, self.k_cache, self.v_cache, batch.table, batch.lens, starts)
        return mol.mol_w4_linear(a.view(x.shape[0], -1), self.out), residual


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
                 block_m=16, group=0, seed=0, heads=0, kv_heads=2, head_dim=128, context=1024, page=16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(g, tokens, H, I, E, k, L, r, block_m, group) for _ in range(layers)]
        self.embed = torch.randn(vocab, H, generator=g, device="cuda").to(torch.bfloat16)
        self.norm = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.head = mol.w4_quantize(torch.randn(vocab, H, generator=g, device="cuda") * H ** -0.5)
        self.batch = Batch(tokens, context, page) if heads else None
        self.attention = [Attention(g, H, heads, kv_heads, head_dim, self.batch) for _ in range(layers)
                          if heads]

    def __call__(self, tokens, lora_ids, counts=None):
        """Logits [T, vocab] of one step: tokens int64 [T], lora_ids int32 [T] (-1: no adapter). With
        attention a token a sequence, or `counts` of them a sequence: its next ones."""
        residual = self.embed[tokens]
        y = torch.zeros_like(residual)
        place = self.batch.place(counts) if self.batch else None
        for i, layer in enumerate(self.layers):
            if self.batch:
                y, residual = self.attention[i](y, residual, self.batch, place)
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
    ap.add_argument("--heads", type=int, default=0, help="query heads of 128, 0 for no attention")
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=0, help="tokens of each sequence before the steps")
    a = ap.parse_args()
    model = Model(tokens=a.tokens, layers=a.layers, group=a.group, heads=a.heads, kv_heads=a.kv_heads,
                  context=a.prompt + a.steps + 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, 5000, (a.tokens,), generator=g, device="cuda")
    lora_ids = torch.randint(-1, 4, (a.tokens,), generator=g, device="cuda").to(torch.int32)
    for _ in range(a.prompt if a.heads else 0):  # (a prompt's chunk is limited by the experts' 128 tokens)
        model(torch.randint(0, 5000, (a.tokens,), generator=g, device="cuda"), lora_ids, [1] * a.tokens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
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
