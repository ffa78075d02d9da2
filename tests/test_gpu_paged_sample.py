"""The operators of a sampled step together, as examples/paged_sample.py uses them: positions, norms and
rotation, rows into the cache, attention, acceptance, commit.

Every accepted node's logits are checked against a plain forward pass over the text so far (causal
attention in float32 over the decoded weights, positions counted from its start): within a fifth of the
row's spread, the bound that test_gpu_paged_verify.py gives the activations' roundings, for both
sides of a difference.  A wrong position, slot, norm or path moves logits by whole spreads.
Each step's paths and bonus tokens are those of the definition in 64 bits on the step's own logits.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_sampled import one_request

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("paged_sample", os.path.join(ROOT, "examples", "paged_sample.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def turned(y, w, freq):
    """Heads [n, heads, D] with their norm and the rotation of halves."""
    y = y / (y.square().mean(2, keepdim=True) + 1e-6).sqrt() * w
    angle = torch.arange(y.shape[0], device="cuda", dtype=torch.float64)[:, None, None] * freq.double()
    a, b = y.chunk(2, 2)
    cos, sin = angle.cos().float(), angle.sin().float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], 2).to(torch.bfloat16).float()


def plain_logits(ex, target, text):
    w = ex.w12.w12_decode
    x = target.embed[torch.tensor(text, device="cuda")]
    n, D, H, G = len(text), target.dim, target.heads, target.q_heads // target.heads
    causal = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
    for l in range(target.layers):
        y = (ex.norm(x).float() @ w(target.qkv[l]).float().T).view(n, -1, D)
        q = turned(y[:, :target.q_heads], target.norms[l][0], target.freq).view(n, H, G, D)
        k = turned(y[:, target.q_heads:target.q_heads + H], target.norms[l][1], target.freq)
        v = y[:, target.q_heads + H:].to(torch.bfloat16).float()
        s = torch.einsum("ihgd,jhd->hgij", q, k) / D ** 0.5
        p = torch.softmax(s.masked_fill(~causal, float("-inf")), -1)
        o = torch.einsum("hgij,jhd->ihgd", p, v).reshape(n, -1).to(torch.bfloat16).float()
        x = x + o @ w(target.out[l]).float().T
    return ex.norm(x).float() @ w(target.head).float().T


@pytest.mark.parametrize("temperature,width,depth,block", [(0.0, 3, 3, 16), (0.8, 3, 2, 8), (1.0, 1, 5, 24), (1.0, 0, 0, 16)])
def test_steps_are_what_the_target_gives(ex, temperature, width, depth, block):
    target = ex.RotatedTarget()
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, 1000, (n,), generator=g).tolist() for n in (1, 7, 300)]
    res = ex.generate(target, prompts, 10, temperature=temperature, block=block, width=width, depth=depth)
    plain = [plain_logits(ex, target, t[:-1]) for t in res.texts]
    at = list(res.prompts)
    for s in res.steps:
        for r in range(3):
            a, b = s.off[r], s.off[r + 1]
            path, bonus = one_request(s.logits[a:b].cpu().numpy(), s.probs[a:b].cpu().numpy(), temperature,
                                      s.parent[a:b].tolist(), s.draft[a:b].tolist(), s.u[a:b].tolist(), float(s.u_bonus[r]))
            assert (s.path_len[r], s.path[a:a + len(path)], s.bonus[r]) == (len(path) - 1, path, bonus)
            for i, node in enumerate(path):
                want = plain[r][at[r] - 1 + i]
                assert float((s.logits[a + node] - want).abs().max()) < 0.2 * float(want.std()), (r, at[r], i)
            assert res.texts[r][at[r]:at[r] + len(path)] == [int(s.draft[a + i]) for i in path[1:]] + [bonus]
            at[r] += len(path)
    if width == 0:
        assert res.accepted == 0


def test_step_in_a_graph(ex):
    """Positions, rows, attention and acceptance captured once with room for more rows than a step has, and
    replayed for another step's trees: the padding's rows are left as they were."""
    w12, dev = ex.w12, "cuda"
    target = ex.RotatedTarget(layers=1)
    R, M, pad, V = 2, 9, 4, target.vocab
    kc, vc = (torch.zeros((1, 64, 16, target.heads, target.dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
    cache, ws, ws2 = w12.KVCache(kc, vc), w12.Workspace(), w12.Workspace()
    table = torch.arange(64, dtype=torch.int32, device=dev).view(2, 32)
    length, off = ex.i32([40, 7]), ex.i32([0, 5, 9])
    parent = ex.i32([-1, 0, 0, 1, 1, -1, 0, 1, 2] + [0] * pad)
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn((M + pad, target.forms[0].width), generator=g, device=dev)
    logits = 3 * torch.randn((M, V), generator=g, device=dev)
    draft = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    u, ub = torch.rand(M, generator=g, device=dev), torch.rand(R, generator=g, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    rows = lambda h: torch.full((M + pad, h, target.dim), 3.0, dtype=torch.bfloat16, device=dev)
    q, k, v = rows(target.q_heads), rows(target.heads), rows(target.heads)

    def step():
        pos, _ = w12.tree_positions(length, parent, off, status=status)
        w12.qkv_rope(x, target.forms[0], pos, q, k, v)
        out, _ = w12.tree_attn(q[:M], k[:M], v[:M], cache, table, length, parent[:M], off, ws=ws, status=status)
        return pos, out, w12.tree_verify_sampled(logits, parent[:M], draft, u, ub, req_offsets=off, ws=ws2, status=status)[:3]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pos, out, accepted = step()
    # another step
    length.copy_(ex.i32([41, 12]))
    off.copy_(ex.i32([0, 3, 9]))
    parent[:M].copy_(ex.i32([-1, 0, 1, -1, 0, 0, 2, 2, 0]))
    for t in (x, logits, u, ub):
        t.copy_(torch.rand(t.shape, generator=g, device=dev))
    for t in (q, k, v):
        t.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (pos, out, q, k, v, *accepted)]
    assert bool((q[M:] == 3).all()) and bool((k[M:] == 3).all()) and bool((v[M:] == 3).all())
    assert pos.tolist() == [41, 42, 43, 12, 13, 13, 14, 14, 13] + [-1] * pad
    pos, out, accepted = step()
    for a, b in zip(got, (pos, out, q, k, v, *accepted)):
        assert torch.equal(a, b)
    assert int(status) == 0
