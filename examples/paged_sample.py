"""Sampled speculative decoding over a paged cache, end to end on one GPU.

    python examples/paged_sample.py [--steps 24] [--requests 3] [--temperature 0.8]

The small random target of paged_verify.py, with norms of the heads and a position rotation.  Every
step drafts a tree per request from a table of next-token probabilities (a stand-in for a drafter),
verifies all trees in one pass and accepts against the target's probabilities:

    tree_positions       the positions of the pass's rows, once for all layers
    kv_append            prompts: q, k and v of every layer, K and V straight into the cache
    qkv_rope             trees: q, k and v of every layer
    tree_attn            attention over the cache and the chunk or tree
    tree_verify_sampled  acceptance and the bonus token from uniform random numbers
    kv_slots, kv_write   the accepted rows into the cache

Whatever the drafter proposes, the text is distributed as if the target had been sampled token by token.
"""
from __future__ import annotations

import argparse
import os
import sys
import typing

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import lossless_bit_weights_gb300 as w12
from examples.paged_verify import CHUNK, Target, i32, norm


class RotatedTarget(Target):
    def __init__(self, seed=0, **kw):
        super().__init__(seed=seed, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        weight = lambda: 1 + 0.2 * torch.randn(self.dim, generator=g, device="cuda")
        self.norms = [(weight(), weight()) for _ in range(self.layers)]
        self.freq = (1e4 ** (-2 * torch.arange(self.dim // 2, device="cuda", dtype=torch.float64) / self.dim)).float()
        self.forms = [w12.QKVForm(self.q_heads, self.heads, self.dim, q_norm=q, k_norm=k, inv_freq=self.freq)
                      for q, k in self.norms]
        # the drafter's table: what the head makes of a token's embedding alone
        self.table = torch.softmax(norm(self.embed).float() @ w12.w12_decode(self.head).float().T, 1)

    def forward(self, tokens, cache, table, cache_len, parent, off, pos, status, slot=None):
        """Logits of every row; with slots K and V go into the cache, else they are returned."""
        x = self.embed[tokens.long()]
        ks, vs = [], []
        for l, form in enumerate(self.forms):
            y = w12.w12_gemm(norm(x), self.qkv[l], ws=self.ws[2 * l])
            if slot is None:
                q, k, v = w12.qkv_rope(y, form, pos)
                ks.append(k)
                vs.append(v)
            else:
                q, k, v, _ = w12.kv_append(y, form, pos, cache, slot, layer=l, rows=True, status=status)
            o, _ = w12.tree_attn(q, k, v, cache, table, cache_len, parent, off, layer=l, ws=self.ws_attn, status=status)
            x = x + w12.w12_gemm(o.flatten(1), self.out[l], ws=self.ws[2 * l + 1])
        logits = w12.w12_gemm(norm(x), self.head, ws=self.ws[-1])
        return (logits, torch.stack(ks), torch.stack(vs)) if slot is None else (logits, None, None)


def draft_tree(table: torch.Tensor, root: int, width: int, depth: int, g: torch.Generator) -> tuple[list[int], list[int]]:
    """Tokens and parents: `width` children of the root, drawn without replacement, each continued by a chain."""
    tok, parent = [root], [-1]
    for t in torch.multinomial(table[root], width, generator=g).tolist() if width else []:
        at = 0
        for _ in range(depth):
            tok.append(t)
            parent.append(at)
            at = len(tok) - 1
            t = int(torch.multinomial(table[t], 1, generator=g))
    return tok, parent


class Step(typing.NamedTuple):
    logits: torch.Tensor
    parent: torch.Tensor
    draft: torch.Tensor
    probs: torch.Tensor
    u: torch.Tensor
    u_bonus: torch.Tensor
    off: list[int]
    path_len: list[int]
    path: list[int]
    bonus: list[int]


class Result(typing.NamedTuple):
    texts: list[list[int]]
    prompts: list[int]
    accepted: float
    steps: list[Step]


def generate(target: RotatedTarget, prompts: list[list[int]], steps: int, temperature: float = 0.8, block: int = 16,
             blocks: int = 512, capacity: int = 4096, width: int = 3, depth: int = 3, seed: int = 0) -> Result:
    R, dev = len(prompts), "cuda"
    kc, vc = (torch.empty((target.layers, blocks, block, target.heads, target.dim), dtype=torch.bfloat16, device=dev)
              for _ in range(2))
    cache = w12.KVCache(kc, vc)
    table = torch.zeros((R, -(-capacity // block)), dtype=torch.int32, device=dev)
    pool, free = torch.arange(blocks, dtype=torch.int32, device=dev), torch.tensor([0, blocks], dtype=torch.int64, device=dev)
    length, status = torch.zeros(R, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    T = torch.full((R,), temperature, device=dev)
    ws, guess = w12.Workspace(), target.table.cpu()
    g, gd = torch.Generator().manual_seed(seed), torch.Generator(device=dev).manual_seed(seed)
    texts, taken, log = [list(p) for p in prompts], 0, []

    # ---- prompts: all tokens but the last, straight into the cache
    at = 0
    while any(len(p) - 1 > at for p in prompts):
        part = [p[at:min(at + CHUNK, len(p) - 1)] for p in prompts]
        off = i32([0] + [sum(len(x) for x in part[:r + 1]) for r in range(R)])
        n = sum(len(x) for x in part)
        s = w12.kv_slots(length, i32([len(x) for x in part]), table, pool, free, block, n, status=status)
        pos, _ = w12.tree_positions(length, req_offsets=off, rows=n, status=status)
        chain = i32([i - 1 for x in part for i in range(len(x))])
        target.forward(i32([t for x in part for t in x]), cache, table, length, chain, off, pos, status, slot=s.slot)
        length, free = s.new_len, s.pool_pos
        at += CHUNK

    # ---- decoding
    for _ in range(steps):
        trees = [draft_tree(guess, t[-1], width, depth, g) for t in texts]
        first = [sum(len(t[0]) for t in trees[:r]) for r in range(R + 1)]
        off, draft, parent = i32(first), i32([t for x in trees for t in x[0]]), i32([p for x in trees for p in x[1]])
        M = draft.numel()
        pos, _ = w12.tree_positions(length, parent, off, status=status)
        logits, k, v = target.forward(draft, cache, table, length, parent, off, pos, status)
        probs = target.table[draft.long()]
        u, ub = torch.rand(M, generator=gd, device=dev), torch.rand(R, generator=gd, device=dev)
        path_len, path, bonus, _ = w12.tree_verify_sampled(logits, parent, draft, u, ub, draft_probs=probs, temperature=T,
                                                           req_offsets=off, ws=ws, status=status)
        s = w12.kv_slots(length, path_len, table, pool, free, block, M, extra=1, path_nodes=path, req_offsets=off, status=status)
        w12.kv_write(cache, k, v, s.slot, src=s.src, status=status)
        length, free = s.new_len, s.pool_pos
        n, nodes, last = path_len.tolist(), path.tolist(), bonus.tolist()
        log.append(Step(logits, parent, draft, probs, u, ub, first, n, nodes, last))
        for r in range(R):
            texts[r] += [trees[r][0][i] for i in nodes[first[r] + 1:first[r] + n[r] + 1]] + [last[r]]
            taken += n[r]
    if int(status):
        raise RuntimeError(f"a call reported status {int(status)}")
    assert length.tolist() == [len(t) - 1 for t in texts]
    return Result(texts, [len(p) for p in prompts], taken / (steps * R), log)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--temperature", type=float, default=0.8)
    a = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1000, (5 + 300 * r,), generator=g).tolist() for r in range(a.requests)]
    res = generate(RotatedTarget(), prompts, a.steps, a.temperature)
    for r, t in enumerate(res.texts):
        new = t[res.prompts[r]:]
        print(f"request {r}: {res.prompts[r]} prompt tokens, {len(new)} new in {a.steps} steps: {new[:12]} ...")
    print(f"accepted drafts a step: {res.accepted:.2f}")


if __name__ == "__main__":
    main()
