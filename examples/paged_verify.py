"""Speculative decoding over a paged cache, end to end on one GPU.

    python examples/paged_verify.py [--steps 24] [--requests 3]

A small random target (W12 projections, attention over a paged cache, a W12 head) serves a
few requests at once.  Every step drafts a tree per request (continuations of earlier
occurrences of the last token in the request's own text, a stand-in for a drafter),
verifies all trees in one pass and commits the accepted paths:

    kv_slots        slots for the prompts, and for each step's accepted path
    tree_attn       every layer's attention over the cache and the tree
    logits_verify   penalties, a bias, a mask of allowed tokens, argmax and acceptance
    kv_write        the accepted rows of all layers into their slots

The prompts go through the same pass, as chains of up to 256 tokens.  Whatever the drafts are,
the text is what one token at a time would give.
"""
from __future__ import annotations

import argparse
import os
import sys
import typing

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import lossless_bit_weights_gb300 as w12

CHUNK = 256  # nodes of a request that one pass takes


def i32(a) -> torch.Tensor:
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def norm(x: torch.Tensor) -> torch.Tensor:
    return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Target:
    """Embedding, layers of attention with a residual, head; no position encoding."""

    def __init__(self, vocab=1000, hidden=512, layers=3, q_heads=6, heads=2, dim=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda n, k, s=1.0: (torch.randn((n, k), generator=g, device="cuda") * s / k ** 0.5).to(torch.bfloat16)
        self.vocab, self.layers, self.q_heads, self.heads, self.dim = vocab, layers, q_heads, heads, dim
        self.embed = torch.randn((vocab, hidden), generator=g, device="cuda")
        self.qkv = [w12.encode(w((q_heads + 2 * heads) * dim, hidden, 1.5)) for _ in range(layers)]
        self.out = [w12.encode(w(hidden, q_heads * dim, 2.0)) for _ in range(layers)]
        self.head = w12.encode(w(vocab, hidden, 3.0))
        self.ws, self.ws_attn = [w12.Workspace() for _ in range(2 * layers + 1)], w12.Workspace()

    def forward(self, tokens, cache, table, cache_len, parent, off, status):
        """Logits of every node and its K and V rows [layers, M, heads, dim]."""
        x = self.embed[tokens.long()]
        a, b = self.q_heads * self.dim, (self.q_heads + self.heads) * self.dim
        ks, vs = [], []
        for l in range(self.layers):
            y = w12.w12_gemm(norm(x), self.qkv[l], ws=self.ws[2 * l]).to(torch.bfloat16)
            q, k, v = (y[:, i:j].unflatten(1, (-1, self.dim)) for i, j in ((0, a), (a, b), (b, y.shape[1])))
            o, _ = w12.tree_attn(q, k, v, cache, table, cache_len, parent, off, layer=l, ws=self.ws_attn, status=status)
            x = x + w12.w12_gemm(o.flatten(1), self.out[l], ws=self.ws[2 * l + 1])
            ks.append(k)
            vs.append(v)
        return w12.w12_gemm(norm(x), self.head, ws=self.ws[-1]), torch.stack(ks), torch.stack(vs)


def draft_tree(text: list[int], width: int, depth: int) -> tuple[list[int], list[int]]:
    """Tokens and parents of a tree below the text's last token: what followed it before, each
    candidate with the token that came after."""
    last = text[-1]
    tok, parent, seen = [last], [-1], set()
    for i in range(len(text) - 2, -1, -1):
        if text[i] != last or text[i + 1] in seen or len(seen) == width:
            continue
        seen.add(text[i + 1])
        at = 0
        for t in text[i + 1:i + 1 + depth]:
            tok.append(t)
            parent.append(at)
            at = len(tok) - 1
    return tok, parent


class Result(typing.NamedTuple):
    texts: list[list[int]]
    prompts: list[int]
    accepted: float
    rules: dict


def generate(target: Target, prompts: list[list[int]], steps: int, block: int = 16, blocks: int = 512, capacity: int = 4096,
             width: int = 3, depth: int = 4, penalties=(1.1, 0.2, 0.1), banned: int = 50, bias: float = 1.0) -> Result:
    R, dev = len(prompts), "cuda"
    kc, vc = (torch.empty((target.layers, blocks, block, target.heads, target.dim), dtype=torch.bfloat16, device=dev)
              for _ in range(2))
    cache = w12.KVCache(kc, vc)
    table = torch.zeros((R, -(-capacity // block)), dtype=torch.int32, device=dev)
    pool, pos = torch.arange(blocks, dtype=torch.int32, device=dev), torch.tensor([0, blocks], dtype=torch.int64, device=dev)
    length, status = torch.zeros(R, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    # rules: the first `banned` tokens are not allowed, token `banned` is a little likelier
    ws, hist = w12.Workspace(), torch.zeros((R, capacity), dtype=torch.int32, device=dev)
    hist_len, prompt_len = torch.zeros_like(length), i32([len(p) for p in prompts])
    rep, freq, pres = (torch.full((R,), v, device=dev) for v in penalties)
    more = (i32(list(range(R + 1))), i32([banned] * R), torch.full((R,), bias, device=dev))
    words = -(-target.vocab // 32)
    allowed = torch.full((words,), -1, dtype=torch.int32, device=dev)
    for t in range(banned):
        allowed[t // 32] &= ~(1 << (t % 32)) if t % 32 < 31 else 0x7FFFFFFF

    texts, taken = [list(p) for p in prompts], 0

    def commit(k, v, path_len, path, off, n):
        nonlocal length, pos
        s = w12.kv_slots(length, path_len, table, pool, pos, block, n, extra=1, path_nodes=path, req_offsets=off, status=status)
        w12.kv_write(cache, k, v, s.slot, src=s.src, status=status)
        length, pos = s.new_len, s.pool_pos

    # ---- prompts: all tokens but the last, which is the first tree's root
    at = 0
    while any(len(p) - 1 > at for p in prompts):
        part = [p[at:min(at + CHUNK, len(p) - 1)] for p in prompts]
        off = i32([0] + [sum(len(x) for x in part[:r + 1]) for r in range(R)])
        parent = i32([i - 1 for x in part for i in range(len(x))])
        _, k, v = target.forward(i32([t for x in part for t in x]), cache, table, length, parent, off, status)
        path = i32([i for x in part for i in range(len(x))])
        commit(k, v, i32([len(x) - 1 for x in part]), path, off, path.numel())
        at += CHUNK

    # ---- decoding
    for _ in range(steps):
        trees = [draft_tree(t, width, depth) for t in texts]
        off = i32([0] + [sum(len(t[0]) for t in trees[:r + 1]) for r in range(R)])
        draft, parent = i32([t for x in trees for t in x[0]]), i32([p for x in trees for p in x[1]])
        M = draft.numel()
        for r, t in enumerate(texts):  # the text before the root
            hist[r, :len(t) - 1] = i32(t[:-1])
        hist_len = i32([len(t) - 1 for t in texts])
        rules = w12.LogitRules(hist=hist, hist_len=hist_len, prompt_len=prompt_len, repetition=rep, frequency=freq,
                               presence=pres, bias=more, mask=allowed.expand(M, words).contiguous())
        logits, k, v = target.forward(draft, cache, table, length, parent, off, status)
        _, path_len, path, bonus, _ = w12.logits_verify(logits, rules, parent, draft, off, ws=ws, status=status)
        commit(k, v, path_len, path, off, M)
        first, n, last, nodes = off.tolist(), path_len.tolist(), bonus.tolist(), path.tolist()
        for r in range(R):
            texts[r] += [trees[r][0][i] for i in nodes[first[r] + 1:first[r] + n[r] + 1]] + [last[r]]
            taken += n[r]
    if int(status):
        raise RuntimeError(f"a call reported status {int(status)}")
    assert length.tolist() == [len(t) - 1 for t in texts]
    return Result(texts, [len(p) for p in prompts], taken / (steps * R),
                  dict(rep=penalties[0], freq=penalties[1], pres=penalties[2], banned=banned, bias=bias))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--requests", type=int, default=3)
    a = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1000, (5 + 300 * r,), generator=g).tolist() for r in range(a.requests)]
    res = generate(Target(), prompts, a.steps)
    for r, t in enumerate(res.texts):
        new = t[res.prompts[r]:]
        print(f"request {r}: {res.prompts[r]} prompt tokens, {len(new)} new in {a.steps} steps: {new[:12]} ...")
    print(f"accepted drafts a step: {res.accepted:.2f}")


if __name__ == "__main__":
    main()
