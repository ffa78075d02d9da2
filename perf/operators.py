"""Cases of the paged-cache operators of a verify step: what is measured and against what.

Five operators work on one step of tree verification over a paged cache: kv_slots (block
tables and slot maps), kv_write (rows into their slots), tree_attn (drafted nodes attend to
the cache and to their ancestors), logits_process (penalties, biases and grammar masks) and
logits_verify (the same with the row argmax and greedy acceptance behind it).  run() makes
either the framework's calls (own) or the plain form: elementary torch operations in 32 bits.
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


def _accepted(case):
    """Accepted path lengths of a commit, or the new prompt tokens, per request."""
    return _spread(case["add_lo"], case["add_hi"], case["requests"])


# ------------------------------------------------------------------ listed cases

def _attn(name, requests, nodes, len_lo, len_hi, hq, hkv, d, block, layout):
    return dict(name=name, op="tree_attn", requests=requests, nodes=nodes, len_lo=len_lo, len_hi=len_hi, hq=hq,
                hkv=hkv, d=d, block=block, layout=layout)


def _slots(name, requests, len_lo, len_hi, add_lo, add_hi, block, commit, release):
    return dict(name=name, op="kv_slots", requests=requests, len_lo=len_lo, len_hi=len_hi, add_lo=add_lo,
                add_hi=add_hi, block=block, commit=commit, release=release)


def _write(name, layers, rows, source_rows, blocks, block, hkv, d):
    return dict(name=name, op="kv_write", layers=layers, rows=rows, source_rows=source_rows, blocks=blocks,
                block=block, hkv=hkv, d=d)


def _logits(name, op, requests, nodes, vocab, hist, penalties, bias, mask):
    return dict(name=name, op=op, requests=requests, nodes=nodes, vocab=vocab, hist=hist, penalties=penalties,
                bias=bias, mask=mask)


def listed():
    return [
        # one request, one token, a short chat: plain decoding, where the call's latency is all
        _attn("attn one token", 1, 1, 711, 711, 40, 8, 128, 16, "nhd"),
        # one request's 16-node tree over a document: the block's 16 rows
        _attn("attn 16-node tree", 1, 16, 8191, 8191, 40, 8, 128, 16, "nhd"),
        # 192 nodes shared by 24 requests of uneven lengths
        _attn("attn 192 nodes, 24 requests", 24, 192, 33, 12001, 40, 8, 128, 32, "nhd"),
        # one long context, wide heads, a 32-node tree, heads outside the tokens in a page
        _attn("attn long context", 1, 32, 131071, 131071, 24, 4, 256, 64, "hnd"),
        # accepted paths of 24 requests get their slots after a step
        _slots("slots of a commit", 24, 33, 12001, -1, 8, 16, True, False),
        # a server admits and releases hundreds of requests at once
        _slots("slots of prompts", 500, 0, 2000, -1, 2047, 16, False, True),
        # the accepted rows of 24 requests into the caches of 16 attention layers
        _write("write of a commit", 16, 101, 192, 512, 16, 8, 128),
        # a batch of prompts into one layer's cache
        _write("write of prompts", 1, 12289, 12289, 1024, 16, 8, 128),
        # one row of one request, short history
        _logits("rules, one row", "logits_process", 1, 1, 32000, 711, True, 3, False),
        # all rules on the rows of 24 requests
        _logits("rules, 192 rows", "logits_process", 24, 192, 151936, 4097, True, 100, True),
        # one tree under a grammar, tokens and acceptance at once
        _logits("verify 16-node tree", "logits_verify", 1, 16, 151936, 8191, True, 20, True),
        # 24 trees with penalties, tokens and acceptance at once
        _logits("verify 192 nodes", "logits_verify", 24, 192, 151936, 2049, True, 20, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree_attn", "tree_attn", "kv_slots", "kv_write", "logits_process", "logits_verify"])
    if op == "tree_attn":
        top = work(listed()[3])
        while True:
            requests = _log(rng, 1, 32)
            d, hkv, group = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
            most = _log(rng, 1, 131072)
            c = _attn("", requests, requests * _log(rng, 1, 64) + rng.randint(0, requests), rng.randint(0, most), most,
                      hkv * group, hkv, d, rng.choice([8, 16, 24, 32, 64, 128]), rng.choice(["nhd", "hnd"]))
            w = work(c)
            # the plain form pads every request to the longest
            pad = requests * hkv * (most + 256) * 4 * (2 * d + 3 * group * (2 + 4 * c["nodes"] // requests))
            if max(_split(c["nodes"], requests)) <= 256 and w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] \
                    and pad < 12e9:
                break
    elif op == "kv_slots":
        commit = rng.random() < 0.5
        requests = _log(rng, 1, 500)
        c = _slots("", requests, 0, _log(rng, 1, 12001), -1 if commit else rng.choice([-1, 0, 1]),
                   rng.randint(1, 16) if commit else _log(rng, 1, 2047), rng.choice([1, 8, 16, 24, 64, 128]), commit,
                   not commit and rng.random() < 0.5)
    elif op == "kv_write":
        layers, hkv, d = rng.choice([1, 1, 2, 7, 16]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        rows = _log(rng, 1, 12289 * 1024 // (layers * hkv * d))
        block = rng.choice([8, 16, 24, 64])
        c = _write("", layers, rows, rows + rng.randint(0, 64), -(-rows // block) + rng.randint(1, 64), block, hkv, d)
    else:
        requests = _log(rng, 1, 24)
        nodes = requests + rng.randint(0, 7 * requests)
        c = _logits("", op, requests, nodes, rng.choice([151936, 32000, 50257, rng.randint(1000, 151936)]),
                    _log(rng, 1, 4097), rng.random() < 0.8, rng.choice([0, 3, 100]), rng.random() < 0.6)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(_DEV)


def _trees(rng, counts):
    """Trees as a drafter grows them: a node hangs under one of the few nodes before it."""
    parent = []
    for n in counts:
        parent += [-1] + [i - 1 - int(min(i, 5) * rng.random() ** 2) for i in range(1, n)]
    return _i32(parent), _i32(np.concatenate([[0], np.cumsum(counts)]))


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=_DEV).manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    {"tree_attn": _prepare_attn, "kv_slots": _prepare_slots, "kv_write": _prepare_write,
     "logits_process": _prepare_logits, "logits_verify": _prepare_logits}[case["op"]](case, rng, g, s)
    return s


def _prepare_attn(c, rng, g, s):
    lens = _spread(c["len_lo"], c["len_hi"], c["requests"])
    counts = _split(c["nodes"], c["requests"])
    s["parent"], s["off"] = _trees(rng, counts)
    s["n_max"] = max(counts)
    need = [-(-n // c["block"]) for n in lens]
    width, blocks = max(1, max(need)), sum(need) + 3
    ids = rng.permutation(blocks)
    table, at = np.zeros((c["requests"], width), np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    s["table"], s["len"] = _i32(table), _i32(lens)
    shape = (blocks, c["block"], c["hkv"], c["d"]) if c["layout"] == "nhd" else (blocks, c["hkv"], c["block"], c["d"])
    kv = [torch.empty(shape, dtype=torch.bfloat16, device=_DEV).normal_(generator=g) for _ in range(2)]
    s["kc"], s["vc"] = kv if c["layout"] == "nhd" else [t.transpose(1, 2) for t in kv]
    # the fused projection's output: q, k and v are strided parts of it
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    qkv = torch.empty((c["nodes"], (hq + 2 * hkv) * d), dtype=torch.bfloat16, device=_DEV).normal_(generator=g)
    qkv[:, :hq * d] *= 2.0  # scores with a spread, as trained heads have them
    s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    if own:
        import lossless_bit_weights_gb300 as w12
        s["cache"] = w12.KVCache(s["kc"], s["vc"])
        s["ws"], s["status"] = w12.Workspace(), torch.zeros(1, dtype=torch.int32, device=_DEV)


def _prepare_slots(c, rng, g, s):
    lens, add = _spread(c["len_lo"], c["len_hi"], c["requests"]), _accepted(c)
    if c["release"]:  # every eighth request has ended
        add = [-1 if r % 8 == 7 else max(a, 0) for r, a in enumerate(add)]
    elif not c["commit"]:
        add = [max(a, 0) for a in add]
    extra = 1 if c["commit"] else 0
    need = [-(-n // c["block"]) for n in lens]
    end = [-(-(n + max(a + extra, 0)) // c["block"]) for n, a in zip(lens, add)]
    free = sum(e - n for e, n in zip(end, need)) + 5
    blocks = sum(need) + free
    ids = rng.permutation(blocks)
    table, at = np.full((c["requests"], max(1, max(end))), -1, np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    head = int(rng.integers(0, blocks))
    pool = np.full(blocks, -1, np.int32)
    pool[(head + np.arange(free)) % blocks] = ids[at:]
    s["table"], s["len"], s["add"], s["pool"] = _i32(table), _i32(lens), _i32(add), _i32(pool)
    s["pos"] = torch.tensor([head, head + free], dtype=torch.int64, device=_DEV)
    s["extra"], s["block"] = extra, c["block"]
    s["capacity"] = sum(max(a + extra, 0) for a in add) + 3  # a fixed launch size, a little above what is used
    s["path"] = s["off"] = None
    if c["commit"]:
        counts = [a + extra + 2 for a in add]
        off = np.concatenate([[0], np.cumsum(counts)])
        path = [np.sort(rng.permutation(n)) for n in counts]
        for p in path:
            p[1:] = np.sort(rng.permutation(np.arange(1, len(p)))) if len(p) > 1 else p[1:]
        s["off"], s["path"] = _i32(off), _i32(np.concatenate(path))
    if own:
        s["status"] = torch.zeros(1, dtype=torch.int32, device=_DEV)


def _prepare_write(c, rng, g, s):
    L, S = c["layers"], c["blocks"] * c["block"]
    shape = (L, c["blocks"], c["block"], c["hkv"], c["d"])
    s["kc"], s["vc"] = [torch.empty(shape, dtype=torch.bfloat16, device=_DEV).normal_(generator=g) for _ in range(2)]
    s["k"], s["v"] = [torch.empty((L, c["source_rows"], c["hkv"], c["d"]), dtype=torch.bfloat16,
                                  device=_DEV).normal_(generator=g) for _ in range(2)]
    s["src"] = _i32(np.sort(rng.permutation(c["source_rows"])[:c["rows"]]))
    # slots come in runs of a block: requests' tokens are neighbours
    ids = rng.permutation(c["blocks"])
    t = np.arange(c["rows"])
    s["slot"] = torch.from_numpy(ids[t // c["block"]] * c["block"] + t % c["block"]).to(_DEV)
    if own:
        import lossless_bit_weights_gb300 as w12
        s["cache"], s["status"] = w12.KVCache(s["kc"], s["vc"]), torch.zeros(1, dtype=torch.int32, device=_DEV)


def _prepare_logits(c, rng, g, s):
    R, M, V = c["requests"], c["nodes"], c["vocab"]
    counts = _split(M, R)
    s["parent"], s["off"] = _trees(rng, counts)
    s["n_max"] = max(counts)
    s["logits"] = torch.empty((M, V), dtype=torch.float32, device=_DEV).normal_(generator=g).mul_(3.0)
    # text: a Zipf-like choice of tokens, spread over the vocabulary
    perm = torch.from_numpy(rng.permutation(V).astype(np.int32)).to(_DEV)

    def words(*shape):
        u = torch.rand(shape, generator=g, device=_DEV)
        return perm[(V ** u - 1).long().clamp_(0, V - 1)]

    s["draft"] = words(M)
    # half the nodes repeat their parent's likeliest token, so that paths are accepted
    base = torch.from_numpy(np.repeat(np.concatenate([[0], np.cumsum(counts)])[:-1], counts)).to(_DEV)
    par = s["parent"].long()
    top = s["logits"].argmax(1).to(torch.int32)
    follow = (torch.rand(M, generator=g, device=_DEV) < 0.5) & (par >= 0)
    s["draft"] = torch.where(follow, top[(base + par).clamp(min=0)], s["draft"])
    s["hist"] = words(R, c["hist"] + 7)
    hl = _spread(max(1, c["hist"] // 8), c["hist"], R)
    s["hist_len"], s["prompt_len"] = _i32(hl), _i32([n // 2 for n in hl])
    s["rep"] = s["freq"] = s["pres"] = None
    if c["penalties"]:
        s["rep"] = 1.0 + 0.3 * torch.rand(R, generator=g, device=_DEV)
        s["freq"] = 0.5 * torch.rand(R, generator=g, device=_DEV)
        s["pres"] = 0.5 * torch.rand(R, generator=g, device=_DEV)
    s["bias"] = None
    if c["bias"]:
        tok = np.concatenate([rng.permutation(V)[:c["bias"]] for _ in range(R)])
        s["bias"] = (_i32(np.arange(R + 1) * c["bias"]), _i32(tok),
                     torch.empty(R * c["bias"], device=_DEV).normal_(generator=g).mul_(4.0))
    s["mask"] = None
    if c["mask"]:  # a grammar allows a few words here, most of the vocabulary there
        words_ = -(-V // 32)
        bits = torch.randint(-2 ** 31, 2 ** 31, (M, words_), generator=g, device=_DEV, dtype=torch.int64)
        thin = torch.randint(-2 ** 31, 2 ** 31, (M, words_), generator=g, device=_DEV, dtype=torch.int64) & \
            torch.randint(-2 ** 31, 2 ** 31, (M, words_), generator=g, device=_DEV, dtype=torch.int64)
        row = (torch.arange(M, device=_DEV) % 3)[:, None]
        s["mask"] = torch.where(row == 0, bits & thin, torch.where(row == 1, bits, bits | thin)).to(torch.int32)
    if own:
        import lossless_bit_weights_gb300 as w12
        s["rules"] = w12.LogitRules(hist=s["hist"], hist_len=s["hist_len"], prompt_len=s["prompt_len"],
                                    repetition=s["rep"], frequency=s["freq"], presence=s["pres"], bias=s["bias"],
                                    mask=s["mask"])
        s["ws"], s["status"] = w12.Workspace(), torch.zeros(1, dtype=torch.int32, device=_DEV)


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"tree_attn": _plain_attn, "kv_slots": _plain_slots, "kv_write": _plain_write,
            "logits_process": _plain_process, "logits_verify": _plain_verify}[s["op"]](s)


def _run_own(s):
    import lossless_bit_weights_gb300 as w12
    op = s["op"]
    if op == "tree_attn":
        return w12.tree_attn(s["q"], s["k"], s["v"], s["cache"], s["table"], s["len"], s["parent"], s["off"],
                             ws=s["ws"], status=s["status"])[0]
    if op == "kv_slots":
        r = w12.kv_slots(s["len"], s["add"], s["table"], s["pool"], s["pos"], s["block"], s["capacity"],
                         extra=s["extra"], path_nodes=s["path"], req_offsets=s["off"], status=s["status"])
        return dict(slot=r.slot, src=r.src, new_len=r.new_len, pool_pos=r.pool_pos, total=r.total, table=s["table"],
                    pool=s["pool"])
    if op == "kv_write":
        w12.kv_write(s["cache"], s["k"], s["v"], s["slot"], src=s["src"], status=s["status"])
        return s["kc"], s["vc"]
    if op == "logits_process":
        return w12.logits_process(s["logits"], s["rules"], s["parent"], s["draft"], s["off"], status=s["status"])[0]
    return w12.logits_verify(s["logits"], s["rules"], s["parent"], s["draft"], s["off"], ws=s["ws"],
                             status=s["status"])[:4]


def _padded(s):
    """Node indices padded to the largest tree: (request, place) -> node, which places hold one, and each
    node's request and place in it."""
    off = s["off"].long()
    n = off[1:] - off[:-1]
    j = torch.arange(s["n_max"], device=_DEV)
    M = s["parent"].shape[0]
    node = (off[:-1, None] + j).clamp(max=M - 1)
    i = torch.arange(M, device=_DEV)
    req = torch.searchsorted(off[1:], i, right=True)
    return node, j < n[:, None], req, i - off[req]


def _ancestors(s, node, held):
    """anc[r, i, j]: node j is on the path from request r's root to its node i."""
    j = torch.arange(s["n_max"], device=_DEV)
    up = (s["parent"].long()[node][..., None] == j) & held[..., None] & held[:, None, :]
    anc = (up | (j[:, None] == j)).float()
    for _ in range(max(1, (s["n_max"] - 1).bit_length())):  # paths of twice the length each time
        anc = (anc @ anc > 0).float()
    return (anc > 0) & held[..., None] & held[:, None, :]


def _plain_attn(s):
    q, k, v, kc, vc = s["q"], s["k"], s["v"], s["kc"], s["vc"]
    node, held, req, place = _padded(s)
    R, n = node.shape
    hkv, d = k.shape[1], k.shape[2]
    G = q.shape[1] // hkv
    anc = _ancestors(s, node, held)
    qp = q[node].float().view(R, n, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, hkv, n * G, d)
    kp = kc[s["table"].long()].flatten(1, 2).permute(0, 2, 3, 1).float()        # R, hkv, d, L
    vp = vc[s["table"].long()].flatten(1, 2).permute(0, 2, 1, 3).float()        # R, hkv, L, d
    L = kp.shape[3]
    scale = 1.0 / math.sqrt(d)
    old = (qp @ kp).mul_(scale).masked_fill_((torch.arange(L, device=_DEV) >= s["len"][:, None])[:, None, None], -math.inf)
    new = (qp @ k[node].float().permute(0, 2, 3, 1)).mul_(scale)
    new = new.masked_fill_(~anc.repeat_interleave(G, 1)[:, None], -math.inf)
    top = torch.maximum(old.amax(3, keepdim=True), new.amax(3, keepdim=True))
    old, new = old.sub_(top).exp_(), new.sub_(top).exp_()
    num = old @ vp + new @ v[node].float().permute(0, 2, 1, 3)
    out = num / (old.sum(3, keepdim=True) + new.sum(3, keepdim=True))
    return out.view(R, hkv, n, G, d).permute(0, 2, 1, 3, 4).reshape(R, n, hkv * G, d)[req, place].to(q.dtype)


def _plain_slots(s):
    block, cap = s["block"], s["pool"].shape[0]
    R, W = s["table"].shape
    lens, a = s["len"].long(), s["add"].long() + s["extra"]
    gone, a = a < 0, a.clamp(min=0)
    have, end = (lens + block - 1) // block, (lens + a + block - 1) // block
    blocks = end - have
    before_blocks, before = blocks.cumsum(0) - blocks, a.cumsum(0) - a
    col = torch.arange(W, device=_DEV)
    table, head, tail = s["table"].clone(), s["pos"][0], s["pos"][1]
    fresh = s["pool"][(head + before_blocks[:, None] + col - have[:, None]) % cap]
    table = torch.where((col >= have[:, None]) & (col < end[:, None]), fresh, table)
    # released blocks go behind the tail
    freed = have * gone
    leave = gone[:, None] & (col < have[:, None])
    at = (tail + (freed.cumsum(0) - freed)[:, None] + col) % cap
    pool = torch.cat([s["pool"], s["pool"][:1]]).scatter_(0, torch.where(leave, at, cap).flatten(), table.flatten())[:cap]
    t = torch.arange(s["capacity"], device=_DEV)
    r = torch.searchsorted(before + a, t, right=True).clamp(max=R - 1)
    used = t < a.sum()
    p = lens[r] + t - before[r]
    slot = torch.where(used, table[r, (p // block).clamp(0, W - 1)].long() * block + p % block, -1)
    if s["path"] is None:
        src = torch.where(used, t, -1).to(torch.int32)
    else:
        o = s["off"].long()[r]
        src = torch.where(used, o + s["path"].long()[(o + t - before[r]).clamp(max=s["path"].shape[0] - 1)], -1).to(torch.int32)
    new_len = torch.where(gone, 0, lens + a).to(torch.int32)
    pos = torch.stack([head + blocks.sum(), tail + freed.sum()])
    return dict(slot=slot, src=src, new_len=new_len, pool_pos=pos, total=a.sum()[None], table=table, pool=pool)


def _plain_write(s):
    L = s["kc"].shape[0]
    for cache, rows in ((s["kc"], s["k"]), (s["vc"], s["v"])):
        cache.view(L, -1, *cache.shape[3:])[:, s["slot"]] = rows[:, s["src"].long()]
    return s["kc"], s["vc"]


def _plain_process(s):
    x = s["logits"]
    M, V = x.shape
    node, held, req, place = _padded(s)
    i = torch.arange(s["hist"].shape[1], device=_DEV)
    hist, one = s["hist"].long(), torch.ones((), device=_DEV)
    live, prompt = i < s["hist_len"][:, None], i < s["prompt_len"][:, None]
    R = hist.shape[0]
    if s["rep"] is not None:
        said = torch.zeros((R, V), device=_DEV).scatter_add_(1, hist, (live & ~prompt).float())
        read = torch.zeros((R, V), device=_DEV).scatter_add_(1, hist, (live & prompt).float())
        anc = _ancestors(s, node, held)[req, place].float()                     # M, n_max
        said = said[req].scatter_add_(1, s["draft"].long()[node][req], anc)     # drafted tokens up to the node
        seen = (said > 0) | (read[req] > 0)
        rep, freq, pres = s["rep"][req, None], s["freq"][req, None], s["pres"][req, None]
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        x = x - freq * said
        x = x - pres * (said > 0).float()
    if s["bias"] is not None:
        _, tok, val = s["bias"]
        b = torch.zeros((R, V), device=_DEV).scatter_(1, tok.long().view(R, -1), val.view(R, -1))
        x = x + b[req]
    if s["mask"] is not None:
        v = torch.arange(V, device=_DEV)
        x = x.masked_fill(((s["mask"][:, v // 32] >> (v % 32)) & 1) == 0, -math.inf)
    return x if x is not s["logits"] else x.clone()


def _plain_verify(s):
    x = _plain_process(s)
    M, V = x.shape
    node, held, req, place = _padded(s)
    # the lowest index of the largest allowed value
    v = torch.arange(V, device=_DEV)
    tok = torch.where(x == x.amax(1, keepdim=True), v, V).amin(1)
    if s["mask"] is not None:
        tok = torch.where((s["mask"] != 0).any(1), tok, -1)
    par = s["parent"].long()
    good = (par < 0) | (tok[(s["off"].long()[req] + par).clamp(min=0)] == s["draft"])
    anc = _ancestors(s, node, held)
    good = (good[node] & held)[:, None, :]
    taken = held & ~(anc & ~good).any(2)
    depth = anc.sum(2) - 1
    j = torch.arange(s["n_max"], device=_DEV)
    length = torch.where(taken, depth, -1).amax(1)
    best = torch.where(taken & (depth == length[:, None]), j, s["n_max"]).amin(1)
    rows = torch.arange(node.shape[0], device=_DEV)
    on = anc[rows, best]
    # node j of the path stands at its depth; -1 behind the path's end
    path = torch.full((node.shape[0], s["n_max"] + 1), -1, device=_DEV, dtype=torch.int64)
    path.scatter_(1, torch.where(on, depth, s["n_max"]), torch.where(on, j, -1))
    return (tok.to(torch.int32), length.to(torch.int32), path[req, place].to(torch.int32),
            tok[node[rows, best]].to(torch.int32))


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    op = c["op"]
    if op == "tree_attn":
        lens, counts = _spread(c["len_lo"], c["len_hi"], c["requests"]), _split(c["nodes"], c["requests"])
        row = 2 * 2 * c["hkv"] * c["d"]                                          # K and V of a token
        b = sum(lens) * row + c["nodes"] * (row + 2 * 2 * c["hq"] * c["d"] + 4) + 4 * sum(-(-n // c["block"]) for n in lens)
        pairs = sum(n * (m + 1) for n, m in zip(counts, lens))                   # the cache and the node itself
        return {"bytes": b, "flops": 4 * c["hq"] * c["d"] * pairs}
    if op == "kv_slots":
        extra = 1 if c["commit"] else 0
        add = [max(a + extra, 0) for a in _accepted(c)]
        lens = _spread(c["len_lo"], c["len_hi"], c["requests"])
        new = sum(-(-(n + a) // c["block"]) - -(-n // c["block"]) for n, a in zip(lens, add))
        touched = sum(-(-(n + a) // c["block"]) - n // c["block"] for n, a in zip(lens, add) if a)
        return {"bytes": 12 * c["requests"] + sum(add) * (12 + (4 if c["commit"] else 0)) + 8 * new + 4 * touched + 32,
                "flops": 0}
    if op == "kv_write":
        return {"bytes": c["layers"] * c["rows"] * c["hkv"] * c["d"] * 2 * 2 * 2 + 12 * c["rows"], "flops": 0}
    M, V = c["nodes"], c["vocab"]
    b = 4 * M * V * (2 if op == "logits_process" else 1) + 8 * M
    b += 4 * sum(_spread(max(1, c["hist"] // 8), c["hist"], c["requests"])) if c["penalties"] else 0
    b += 8 * c["bias"] * c["requests"] + (4 * M * -(-V // 32) if c["mask"] else 0)
    return {"bytes": b, "flops": M * V}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "kv_slots":
        return None
    if op == "kv_write":
        out = []
        for cache, rows in ((s["kc"], s["k"]), (s["vc"], s["v"])):
            c = cache.double()
            for t, (a, b) in enumerate(zip(s["slot"].tolist(), s["src"].tolist())):
                c[:, a // case["block"], a % case["block"]] = rows[:, b].double()
            out.append(c)
        return tuple(out)
    off, parent = s["off"].tolist(), s["parent"].tolist()

    def path(r, i):
        p = []
        while i >= 0:
            p.append(i)
            i = parent[off[r] + i]
        return p[::-1]

    if op == "tree_attn":
        G = case["hq"] // case["hkv"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=_DEV)
        for r, n in enumerate(s["len"].tolist()):
            ids = s["table"][r, :-(-n // case["block"])].long()
            K, V = (t[ids].reshape(-1, *t.shape[2:])[:n].double() for t in (s["kc"], s["vc"]))
            mine = slice(off[r], off[r + 1])
            m = off[r + 1] - off[r]
            K, V = torch.cat([K, s["k"][mine].double()]), torch.cat([V, s["v"][mine].double()])
            may = torch.zeros((m, n + m), dtype=torch.bool)
            may[:, :n] = True
            for i in range(m):
                may[i, [n + j for j in path(r, i)]] = True
            may = may.to(_DEV)
            for h in range(case["hq"]):
                z = s["q"][mine, h].double() @ K[:, h // G].T / math.sqrt(case["d"])
                z[~may] = -math.inf
                out[mine, h] = torch.softmax(z, 1) @ V[:, h // G]
        return out
    x = s["logits"].double()
    M, V = x.shape
    hist, draft = s["hist"].tolist(), s["draft"].tolist()
    hl, pl = s["hist_len"].tolist(), s["prompt_len"].tolist()
    for r in range(case["requests"]):
        out0 = torch.bincount(torch.tensor(hist[r][pl[r]:hl[r]], dtype=torch.int64), minlength=V)
        in0 = torch.bincount(torch.tensor(hist[r][:pl[r]], dtype=torch.int64), minlength=V)
        for i in range(off[r], off[r + 1]):
            n = out0.clone()
            for j in path(r, i - off[r]):
                n[draft[off[r] + j]] += 1
            if s["rep"] is not None:
                m = ((n > 0) | (in0 > 0)).to(_DEV)
                n = n.to(_DEV).double()
                rep, fr, pr = (s[w][r].double() for w in ("rep", "freq", "pres"))
                x[i] = torch.where(m, torch.where(x[i] > 0, x[i] / rep, x[i] * rep), x[i]) - fr * n - pr * (n > 0)
            if s["bias"] is not None:
                o, tok, val = s["bias"]
                mine = slice(int(o[r]), int(o[r + 1]))
                x[i, tok[mine].long()] += val[mine].double()
            if s["mask"] is not None:
                words = s["mask"][i].cpu().numpy().view(np.uint8)
                allowed = np.unpackbits(words, bitorder="little")[:V].astype(bool)
                x[i][~torch.from_numpy(allowed).to(_DEV)] = -math.inf
    if op == "logits_process":
        return x
    return None  # tokens and paths are whole numbers
