"""Cases of the operators of a sampled verify step: what is measured and against what.

tree_positions gives every node of the draft trees its position; qkv_rope turns the fused
projection's rows into q, k and v (norms of each head, position rotation); kv_append does the
same for tokens that need no acceptance and puts K and V straight into the paged cache;
tree_verify_sampled accepts drafted tokens against the target's probabilities from given random
numbers.  run() makes either the framework's calls (own) or the plain form: elementary torch
operations in 32 bits, the angles, sums and decisions in 64.
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda"
_PHI = 0.6180339887498949


# ------------------------------------------------------------------ sizes that follow from a case alone

def _spread(lo, hi, n):
    """n sizes over lo..hi, the first one hi (golden-ratio steps, so no two neighbours are alike)."""
    return [hi - int((hi - lo) * ((i * _PHI) % 1.0)) for i in range(n)]


def _split(total, n):
    """total nodes over n requests, at least one each, unevenly."""
    w = np.cumsum([1.0 + 3.0 * ((i * _PHI) % 1.0) for i in range(n)])
    off = np.floor((total - n) * w / w[-1]).astype(np.int64) + np.arange(1, n + 1)
    off[-1] = total
    return np.diff(np.concatenate([[0], off])).tolist()


# ------------------------------------------------------------------ listed cases

def _pos(name, requests, nodes, len_lo, len_hi, tree, pad):
    return dict(name=name, op="tree_positions", requests=requests, nodes=nodes, len_lo=len_lo, len_hi=len_hi, tree=tree,
                pad=pad)


def _rope(name, rows, pos_hi, hq, hkv, d, rot, pairs, norm, kind):
    return dict(name=name, op="qkv_rope", rows=rows, pos_hi=pos_hi, hq=hq, hkv=hkv, d=d, rot=rot, pairs=pairs, norm=norm,
                kind=kind)


def _append(name, rows, pad, pos_hi, hq, hkv, d, rot, pairs, norm, kind, block, layout, keep):
    return dict(name=name, op="kv_append", rows=rows, pad=pad, pos_hi=pos_hi, hq=hq, hkv=hkv, d=d, rot=rot, pairs=pairs,
                norm=norm, kind=kind, block=block, layout=layout, keep=keep)


def _sampled(name, requests, nodes, vocab, shape, probs, temperature):
    return dict(name=name, op="tree_verify_sampled", requests=requests, nodes=nodes, vocab=vocab, shape=shape, probs=probs,
                temperature=temperature)


def listed():
    return [
        # the nodes of 24 requests' trees, once a step
        _pos("positions of 24 trees", 24, 192, 33, 12001, True, 5),
        # prompts of hundreds of requests, admitted at once
        _pos("positions of prompts", 500, 448507, 0, 12001, False, 64),
        # one token of one request: the call's latency is all
        _rope("rope, one row", 1, 711, 40, 8, 128, 128, "halves", True, "float"),
        # the rows of 24 requests' trees in one layer, as the projection leaves them
        _rope("rope, 192 rows", 192, 12009, 40, 8, 128, 128, "halves", True, "float"),
        # a batch of prompts: wide heads rotated in part, adjacent pairs, no norms, bf16 rows
        _rope("rope of prompts", 12289, 131071, 24, 4, 256, 64, "adjacent", False, "bf16"),
        # plain decoding of 24 requests in a captured graph of 32 rows
        _append("append one token each", 24, 8, 12001, 40, 8, 128, 128, "halves", True, "float", 16, "nhd", True),
        # one request's chunk of a prompt, rows kept for the attention among them
        _append("append a chunk", 256, 0, 8191, 40, 8, 128, 128, "halves", True, "float", 64, "hnd", True),
        # a batch of prompts into the cache, float rows
        _append("append prompts", 12289, 0, 12289, 40, 8, 128, 128, "halves", True, "float", 16, "nhd", False),
        # a token of one request, nothing drafted: plain sampling
        _sampled("sample one row", 1, 1, 32000, "tree", False, True),
        # one request's 16-node tree with the drafter's probabilities
        _sampled("sampled 16-node tree", 1, 16, 151936, "tree", True, True),
        # 24 requests' trees with the drafter's probabilities
        _sampled("sampled 192 nodes", 24, 192, 151936, "tree", True, True),
        # chains of 4 drafts for 64 requests from a drafter that gives tokens alone
        _sampled("sampled chains", 64, 320, 151936, "chain", False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    d, hkv, group = rng.choice([64, 96, 128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
    rot = rng.choice([d, d, d // 2, 32])
    return dict(hq=hkv * group, hkv=hkv, d=d, rot=rot, pairs=rng.choice(["halves", "adjacent"]), norm=rng.random() < 0.6,
                kind=rng.choice(["float", "bf16"]))


def draw(rng):
    op = rng.choice(["tree_positions", "qkv_rope", "kv_append", "tree_verify_sampled", "tree_verify_sampled"])
    top = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        if op == "tree_positions":
            tree, requests = rng.random() < 0.6, _log(rng, 1, 500)
            nodes = requests * _log(rng, 1, 64 if tree else 897) + rng.randint(0, requests)
            c = _pos("", requests, nodes, 0, _log(rng, 1, 131071), tree, rng.choice([0, 5, 64]))
        elif op == "qkv_rope":
            c = _rope("", _log(rng, 1, 12289), _log(rng, 64, 1048575), **_heads(rng))
        elif op == "kv_append":
            c = _append("", _log(rng, 1, 12289), rng.choice([0, 0, 8]), _log(rng, 64, 1048575), **_heads(rng),
                        block=rng.choice([8, 16, 24, 64]), layout=rng.choice(["nhd", "hnd"]), keep=rng.random() < 0.5)
        else:
            requests = _log(rng, 1, 64)
            nodes = requests + rng.randint(0, 7 * requests) if requests > 1 else _log(rng, 1, 64)
            c = _sampled("", requests, nodes, rng.choice([151936, 32000, 50257, rng.randint(1000, 151936)]),
                         rng.choice(["tree", "tree", "chain"]), rng.random() < 0.6, rng.random() < 0.7)
        if work(c)["bytes"] <= top and c.get("nodes", 0) * c.get("vocab", 0) <= 320 * 151936:
            del c["name"]
            return c


# ------------------------------------------------------------------ inputs

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(_DEV)


def _trees(rng, counts, chain=False):
    """Trees as a drafter grows them: a node hangs under one of the few nodes before it."""
    parent = []
    for n in counts:
        parent += [-1] + [i - 1 - (0 if chain else int(min(i, 5) * rng.random() ** 2)) for i in range(1, n)]
    return np.asarray(parent, np.int64), np.concatenate([[0], np.cumsum(counts)])


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=_DEV).manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    {"tree_positions": _prepare_positions, "qkv_rope": _prepare_rope, "kv_append": _prepare_append,
     "tree_verify_sampled": _prepare_sampled}[case["op"]](case, rng, g, s)
    if own:
        s["status"] = torch.zeros(1, dtype=torch.int32, device=_DEV)
    return s


def _prepare_positions(c, rng, g, s):
    counts = _split(c["nodes"], c["requests"])
    parent, off = _trees(rng, counts)
    s["parent"] = _i32(np.concatenate([parent, np.full(c["pad"], -1)])) if c["tree"] else None
    s["off"], s["rows"], s["n_max"] = _i32(off), c["nodes"] + c["pad"], max(counts)
    s["len"] = _i32(rng.permutation(_spread(c["len_lo"], c["len_hi"], c["requests"])))


def _rows_of_projection(c, rows, g, s):
    """The fused projection's rows, the norms' weights and the frequencies."""
    width = (c["hq"] + 2 * c["hkv"]) * c["d"]
    x = torch.empty((rows, width), dtype=torch.float32, device=_DEV).normal_(generator=g)
    x *= torch.exp2(torch.empty((rows, 1), device=_DEV).normal_(generator=g))  # rows of unlike sizes
    s["x"] = x if c["kind"] == "float" else x.to(torch.bfloat16)
    s["wq"], s["wk"] = [torch.empty(c["d"], device=_DEV).normal_(generator=g).mul_(0.2).add_(1.0) if c["norm"] else None
                        for _ in range(2)]
    j = torch.arange(c["rot"] // 2, dtype=torch.float64, device=_DEV)
    s["freq"] = (1e6 ** (-2.0 * j / c["rot"])).float()
    s["eps"] = 1e-6
    if own:
        import lossless_bit_weights_gb300 as w12
        s["form"] = w12.QKVForm(c["hq"], c["hkv"], c["d"], q_norm=s["wq"], k_norm=s["wk"], eps=s["eps"], inv_freq=s["freq"],
                                interleaved=c["pairs"] == "adjacent")


def _prepare_rope(c, rng, g, s):
    _rows_of_projection(c, c["rows"], g, s)
    s["pos"] = _i32(rng.integers(0, c["pos_hi"] + 1, c["rows"]))


def _prepare_append(c, rng, g, s):
    n, rows = c["rows"], c["rows"] + c["pad"]
    _rows_of_projection(c, rows, g, s)
    block, hkv, d = c["block"], c["hkv"], c["d"]
    blocks = -(-n // block) + 5
    shape = (2, blocks, block, hkv, d) if c["layout"] == "nhd" else (2, blocks, hkv, block, d)
    kv = [torch.empty(shape, dtype=torch.bfloat16, device=_DEV).normal_(generator=g) for _ in range(2)]
    s["kc"], s["vc"] = kv if c["layout"] == "nhd" else [t.transpose(2, 3) for t in kv]
    # slots come in runs of a block: requests' tokens are neighbours; the rows behind the tokens are a graph's padding
    ids, t = rng.permutation(blocks), np.arange(n)
    pad = np.full(c["pad"], -1)
    s["slot"] = torch.from_numpy(np.concatenate([ids[t // block] * block + t % block, pad])).to(_DEV)
    s["pos"] = _i32(np.concatenate([(rng.integers(0, c["pos_hi"] + 1) + t) % (c["pos_hi"] + 1), pad]))
    new = lambda heads: torch.zeros((rows, heads, d), dtype=torch.bfloat16, device=_DEV)
    s["q"], s["k"], s["v"] = new(c["hq"]), new(hkv) if c["keep"] else None, new(hkv) if c["keep"] else None
    if own:
        import lossless_bit_weights_gb300 as w12
        s["cache"] = w12.KVCache(s["kc"], s["vc"])


def _prepare_sampled(c, rng, g, s):
    R, M, V = c["requests"], c["nodes"], c["vocab"]
    counts = _split(M, R)
    parent, off = _trees(rng, counts, c["shape"] == "chain")
    s["parent"], s["off"], s["n_max"] = _i32(parent), _i32(off), max(counts)
    s["logits"] = torch.empty((M, V), dtype=torch.float32, device=_DEV).normal_(generator=g).mul_(3.0)
    # a few tokens stand out of the many, as a trained target has them
    few = torch.randint(0, V, (M, 8), generator=g, device=_DEV)
    s["logits"].scatter_(1, few, 12.0 + 8.0 * torch.rand((M, 8), generator=g, device=_DEV))
    s["temperature"] = None
    if c["temperature"]:  # every eighth request asks for the likeliest tokens
        s["temperature"] = (0.6 + 0.6 * torch.rand(R, generator=g, device=_DEV)) * (torch.arange(R, device=_DEV) % 8 != 7)
    # the drafter: what the target thinks, and its own mistakes
    guess = 0.9 * s["logits"] + torch.empty((M, V), dtype=torch.float32, device=_DEV).normal_(generator=g).mul_(0.8)
    if c["temperature"]:
        t = torch.where(s["temperature"] > 0, s["temperature"], 1.0)
        guess /= t.repeat_interleave(torch.tensor(counts, device=_DEV))[:, None]
    guess = torch.log_softmax(guess, 1)
    s["probs"] = guess.exp() if c["probs"] else None
    # the children of a node are its likeliest tokens under a Gumbel perturbation: draws without
    # replacement; a drafter that gives tokens alone takes its likeliest ones
    base = np.repeat(off[:-1], counts)
    rank, seen = np.zeros(M, np.int64), {}
    for i in range(M):
        k = (base[i], parent[i])
        rank[i] = seen[k] = seen.get(k, -1) + 1 if parent[i] >= 0 else 0
    if c["probs"]:
        guess -= torch.log(-torch.log(torch.rand((M, V), generator=g, device=_DEV).clamp_(1e-7, 1 - 1e-7)))
    best = guess.topk(int(rank.max()) + 1, 1).indices
    up = torch.from_numpy(np.maximum(base + parent, 0)).to(_DEV)
    s["draft"] = best[up, torch.from_numpy(rank).to(_DEV)].to(torch.int32)
    s["u"], s["u_bonus"] = torch.rand(M, generator=g, device=_DEV), torch.rand(R, generator=g, device=_DEV)
    if own:
        import lossless_bit_weights_gb300 as w12
        s["ws"] = w12.Workspace()


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"tree_positions": _plain_positions, "qkv_rope": _plain_rope, "kv_append": _plain_append,
            "tree_verify_sampled": _plain_sampled}[s["op"]](s)


def _run_own(s):
    import lossless_bit_weights_gb300 as w12
    op = s["op"]
    if op == "tree_positions":
        return w12.tree_positions(s["len"], s["parent"], s["off"], rows=s["rows"], status=s["status"])[0]
    if op == "qkv_rope":
        return w12.qkv_rope(s["x"], s["form"], s["pos"])
    if op == "kv_append":
        w12.kv_append(s["x"], s["form"], s["pos"], s["cache"], s["slot"], layer=1, q=s["q"], k=s["k"], v=s["v"],
                      status=s["status"])
        return [t for t in (s["q"], s["k"], s["v"]) if t is not None] + [s["kc"], s["vc"]]
    return w12.tree_verify_sampled(s["logits"], s["parent"], s["draft"], s["u"], s["u_bonus"], draft_probs=s["probs"],
                                   temperature=s["temperature"], req_offsets=s["off"], ws=s["ws"], status=s["status"])[:3]


def _place(s, rows):
    """Each row's request (a last one for the rows behind all requests) and place in it."""
    off = s["off"].long()
    i = torch.arange(rows, device=_DEV)
    req = torch.searchsorted(off[1:], i, right=True)
    return req, i - off[req]


def _plain_positions(s):
    rows = s["rows"]
    req, place = _place(s, rows)
    start = torch.cat([s["len"].long(), s["len"].new_zeros(1).long()])[req]
    if s["parent"] is None:
        depth = place
    else:
        i = torch.arange(rows, device=_DEV)
        up = torch.where(s["parent"] >= 0, i - place + s["parent"].long(), i)
        depth = (up != i).long()
        for _ in range(max(1, (s["n_max"] - 1).bit_length())):  # twice as far up each time
            depth, up = depth + depth[up], up[up]
    return torch.where(req < s["len"].shape[0], start + depth, -1).to(torch.int32)


def _rotated(s):
    c = s["case"]
    d, half = c["d"], c["rot"] // 2
    x = s["x"].float().unflatten(1, (-1, d))
    parts = list(x.split([c["hq"], c["hkv"], c["hkv"]], 1))
    angle = s["pos"].double()[:, None, None] * s["freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    for i, w in enumerate((s["wq"], s["wk"])):
        y = parts[i]
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(2, keepdim=True) + s["eps"]) * w
        if c["pairs"] == "halves":
            a, b, rest = y[..., :half], y[..., half:2 * half], y[..., 2 * half:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin, rest], 2)
        else:
            a, b, rest = y[..., 0:2 * half:2], y[..., 1:2 * half:2], y[..., 2 * half:]
            y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2), rest], 2)
        parts[i] = y
    return [p.to(torch.bfloat16) for p in parts]


def _plain_rope(s):
    return tuple(_rotated(s))


def _plain_append(s):
    rows = _rotated(s)
    live, slot = s["pos"] >= 0, s["slot"].clamp(min=0)
    for out, y in zip((s["q"], s["k"], s["v"]), rows):
        if out is not None:
            out.copy_(torch.where(live[:, None, None], y, out))
    n = s["case"]["rows"]  # the tokens stand before the padding
    block = s["case"]["block"]
    for cache, y in ((s["kc"], rows[1]), (s["vc"], rows[2])):
        cache[1].index_put_((slot[:n] // block, slot[:n] % block), y[:n])
    return [t for t in (s["q"], s["k"], s["v"]) if t is not None] + [s["kc"], s["vc"]]


def _plain_sampled(s):
    """Node after node in index order, all requests at once: a node whose parent is the last accepted one is
    tested; refused, it changes what is left of the probabilities."""
    x, off, parent = s["logits"], s["off"].long(), s["parent"].long()
    M, V = x.shape
    R = off.shape[0] - 1
    one = torch.arange(V, device=_DEV)
    T = s["temperature"].double()[:, None] if s["temperature"] is not None else torch.ones((R, 1), dtype=torch.float64, device=_DEV)
    greedy = T < 1e-5

    def target(rows):
        l = x[rows]
        most = l.amax(1, keepdim=True)
        first = torch.where(l == most, one, V).amin(1, keepdim=True)
        e = ((l.double() - most.double()) / torch.where(greedy, 1.0, T)).exp_()
        return torch.where(greedy, (one == first).double(), e / e.sum(1, keepdim=True))

    def drafted(rows):
        return s["probs"][rows].double() if s["probs"] is not None else None

    p, q, Q = target(off[:-1]), drafted(off[:-1]), torch.ones((R, 1), dtype=torch.float64, device=_DEV)
    cur, depth = torch.zeros(R, dtype=torch.int64, device=_DEV), torch.zeros(R, dtype=torch.int64, device=_DEV)
    path = torch.full((M + 1,), -1, dtype=torch.int32, device=_DEV)
    path[off[:-1]] = 0
    for j in range(1, s["n_max"]):
        i = (off[:-1] + j).clamp(max=M - 1)
        child = (off[:-1] + j < off[1:]) & (parent[i] == cur)
        t = s["draft"][i].long()[:, None]
        px = p.gather(1, t)
        qx = q.gather(1, t) if q is not None else torch.ones_like(px)
        take = child & (s["u"][i].double() * (qx / Q)[:, 0] < px[:, 0])
        miss = (child & ~take)[:, None]
        left = (p - q / Q).clamp_(min=0) if q is not None else p.scatter(1, t, 0.0)
        p = torch.where(miss, left / left.sum(1, keepdim=True), p)
        if q is not None:
            Q = torch.where(miss, Q - qx, Q)
            q = torch.where(miss, q.scatter(1, t, 0.0), q)
            q = torch.where(take[:, None], drafted(i), q)
        Q = torch.where(take[:, None], 1.0, Q)
        p = torch.where(take[:, None], target(i), p)
        cur = torch.where(take, j, cur)
        depth = depth + take
        path[torch.where(take, off[:-1] + depth, M)] = j
    cdf = p.cumsum(1)
    bonus = (cdf <= s["u_bonus"].double()[:, None] * cdf[:, -1:]).sum(1)
    return depth.to(torch.int32), path[:M], bonus.to(torch.int32)


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    op = c["op"]
    if op == "tree_positions":
        return {"bytes": 4 * (c["nodes"] + c["pad"]) + (4 * c["nodes"] if c["tree"] else 0) + 8 * c["requests"] + 4,
                "flops": 0}
    if op == "tree_verify_sampled":
        # the rows of the accepted path's nodes, of which each step adds one with a chance of about 0.6 (without
        # probabilities 0.45, as measured on these inputs), and the drafter's row where the path ends above other drafts
        n, a = c["nodes"] / c["requests"], 0.6 if c["probs"] else 0.45
        most = n if c["shape"] == "chain" else 1 + 0.7 * (n - 1)
        visited = (1 - a ** most) / (1 - a)
        rows = visited + (1.0 if c["probs"] and n > 1 else 0.0)
        return {"bytes": int(4 * c["requests"] * c["vocab"] * rows) + 16 * c["nodes"] + 20 * c["requests"],
                "flops": int(10 * c["requests"] * c["vocab"] * rows)}
    rows, d = c["rows"], c["d"]
    size = 4 if c["kind"] == "float" else 2
    heads = c["hq"] + 2 * c["hkv"]
    b = rows * heads * d * (size + 2) + 4 * rows + 2 * c["rot"] + (8 * d if c["norm"] else 0)
    if op == "kv_append":
        b += 12 * c["pad"] + 8 * rows + (rows * 2 * c["hkv"] * d * 2 if c["keep"] else 0)
    return {"bytes": b, "flops": rows * ((c["hq"] + c["hkv"]) * ((4 * d if c["norm"] else 0) + 3 * c["rot"]) + 10 * c["rot"])}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("tree_positions", "tree_verify_sampled"):
        return None  # positions, paths and tokens are whole numbers
    s = prepare(case, seed)
    d, rot, hq, hkv = case["d"], case["rot"], case["hq"], case["hkv"]
    x = s["x"].double()
    # each rotated pair as a complex number
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=_DEV).expand(x.shape[0], rot // 2),
                       s["pos"].double()[:, None] * s["freq"].double())
    if case["pairs"] == "halves":
        first, second = torch.arange(rot // 2, device=_DEV), torch.arange(rot // 2, rot, device=_DEV)
    else:
        first, second = torch.arange(0, rot, 2, device=_DEV), torch.arange(1, rot, 2, device=_DEV)
    out = []
    for h in range(hq + 2 * hkv):
        y = x[:, h * d:(h + 1) * d].clone()
        if h < hq + hkv:
            w = s["wq"] if h < hq else s["wk"]
            if w is not None:
                y = w.double() * y / ((y * y).sum(1, keepdim=True) / d + s["eps"]).sqrt()
            z = torch.complex(y[:, first], y[:, second]) * turn
            y[:, first], y[:, second] = z.real, z.imag
        out.append(y)
    out = torch.stack(out, 1)
    rows = [out[:, :hq], out[:, hq:hq + hkv], out[:, hq + hkv:]]
    if op == "qkv_rope":
        return tuple(rows)
    n = case["rows"]
    caches = []
    for cache, y in ((s["kc"], rows[1]), (s["vc"], rows[2])):
        c = cache.double()
        for t, a in enumerate(s["slot"][:n].tolist()):
            c[1, a // case["block"], a % case["block"]] = y[t]
        caches.append(c)
    kept = [torch.where((s["pos"] >= 0)[:, None, None], y, 0.0) for y in (rows if case["keep"] else rows[:1])]
    return kept + caches
