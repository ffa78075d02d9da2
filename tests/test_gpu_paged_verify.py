"""The paged-cache operators together, as examples/paged_verify.py uses them.

Every token of the generated texts is checked against a plain forward pass over the whole
text (causal attention in float32 over the decoded weights): its value under the rules is within
a tenth of the row's spread of the largest one.  (The activations' roundings to bf16 fall
elsewhere in passes of other sizes, so near-ties may differ; a wrong slot, mask, count or
path moves values by whole spreads.)
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("paged_verify", os.path.join(ROOT, "examples", "paged_verify.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_logits(ex, target, text):
    w = ex.w12.w12_decode
    x = target.embed[torch.tensor(text, device="cuda")]
    n, D, G = len(text), target.dim, target.q_heads // target.heads
    causal = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
    for l in range(target.layers):
        y = (ex.norm(x).float() @ w(target.qkv[l]).float().T).to(torch.bfloat16).float()
        q = y[:, :target.q_heads * D].view(n, target.heads, G, D)
        k, v = y[:, target.q_heads * D:].view(n, 2, target.heads, D).unbind(1)
        s = torch.einsum("ihgd,jhd->hgij", q, k) / D ** 0.5
        p = torch.softmax(s.masked_fill(~causal, float("-inf")), -1)
        o = torch.einsum("hgij,jhd->ihgd", p, v).reshape(n, -1).to(torch.bfloat16).float()
        x = x + o @ w(target.out[l]).float().T
    return ex.norm(x).float() @ w(target.head).float().T


def under_rules(res, r, logits, text, i):
    """Row i (the prediction after text[i]) under the rules."""
    x, n = logits[i].clone(), torch.zeros(logits.shape[1], device="cuda")
    for t in text[res.prompts[r]:i + 1]:
        n[t] += 1
    seen = n > 0
    seen[torch.tensor(text[:min(res.prompts[r], i)], dtype=torch.long, device="cuda")] = True
    if i < res.prompts[r]:  # the prompt's last token is the first root: drafted, so it counts
        n[text[i]] += 1
        seen[text[i]] = True
    x = torch.where(seen, torch.where(x > 0, x / res.rules["rep"], x * res.rules["rep"]), x)
    x = x - res.rules["freq"] * n - res.rules["pres"] * (n > 0).float()
    x[res.rules["banned"]] += res.rules["bias"]
    x[:res.rules["banned"]] = float("-inf")
    return x


@pytest.mark.parametrize("width,depth", [(0, 0), (1, 6), (4, 3)])
@pytest.mark.parametrize("block", [8, 24])
def test_texts_are_what_one_token_at_a_time_gives(ex, width, depth, block):
    target = ex.Target()
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, 1000, (n,), generator=g).tolist() for n in (1, 7, 300)]
    res = ex.generate(target, prompts, 16, block=block, width=width, depth=depth)
    for r, text in enumerate(res.texts):
        assert len(text) >= res.prompts[r] + 16
        logits = plain_logits(ex, target, text[:-1])
        for i in range(res.prompts[r] - 1, len(text) - 1):
            x = under_rules(res, r, logits, text, i)
            fin = x[torch.isfinite(x)]
            assert x[text[i + 1]] >= fin.max() - 0.1 * fin.std(), (r, i)
    if width == 0:
        assert res.accepted == 0


def test_drafts_are_accepted(ex):
    """Without penalties a text soon repeats itself; its own continuations are then right."""
    res = ex.generate(ex.Target(), [[7, 8, 9], [500] * 40], 30, penalties=(1.0, 0.0, 0.0))
    assert res.accepted > 0.3


def test_the_prompt_is_not_penalised_as_output(ex):
    """A token with a large bias is the first one generated although the prompt ends with it, and not the
    second, which is penalised for the first."""
    res = ex.generate(ex.Target(), [[50], [3, 50], [50, 7, 50]], 2, penalties=(1.0, 15.0, 15.0), banned=50, bias=20.0)
    for r, text in enumerate(res.texts):
        assert text[res.prompts[r]] == 50 and text[res.prompts[r] + 1] != 50
