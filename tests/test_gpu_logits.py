"""logits_process and logits_verify against a plain implementation.

The formula is a few float operations per token, each rounded, so the processed logits are
compared bit for bit with the same operations in numpy's float32, and with the formula in 64
bits within 8 roundings (2^-21) of the largest term.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lossless_bit_weights_gb300 as m
    m.lib()
    return m


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.float32))).cuda()


class Problem:
    def __init__(self, seed, counts, V, hist=50, penalties=("rep", "freq", "pres"), bias=5, mask="half", words=None):
        rng = np.random.default_rng(seed)
        self.counts, self.V = counts, V
        R, M = len(counts), int(sum(counts))
        self.off = np.concatenate([[0], np.cumsum(counts)])
        self.parents = [[-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)] if n else [] for n in counts]
        self.logits = (rng.standard_normal((M, V)) * 3).astype(np.float32)
        few = rng.integers(0, V, max(1, min(V, 30)))     # tokens repeat
        self.draft = rng.choice(few, M).astype(np.int32)
        self.hist = rng.choice(few, (R, hist + 3)).astype(np.int32)
        self.hist_len = rng.integers(0, hist + 1, R).astype(np.int32)
        self.prompt_len = np.array([rng.integers(0, n + 1) for n in self.hist_len], np.int32)
        u = lambda lo, hi: rng.uniform(lo, hi, R).astype(np.float32)
        self.pen = {"rep": u(1.0, 1.5), "freq": u(-0.3, 0.5), "pres": u(-0.3, 0.5)}
        self.pen = {k: v for k, v in self.pen.items() if k in penalties}
        self.bias = None
        if bias:
            n = [int(rng.integers(0, bias + 1)) for _ in range(R)]
            n[0] = bias
            self.bias = (np.concatenate([[0], np.cumsum(n)]).astype(np.int32),
                         rng.integers(0, V, sum(n)).astype(np.int32), (rng.standard_normal(sum(n)) * 4).astype(np.float32))
        self.allowed = None
        if mask:
            self.words = words or -(-V // 32)
            bits = rng.random((M, self.words * 32)) < {"half": 0.5, "thin": 0.01, "none": 0.0}[mask]
            self.allowed = bits[:, :V]
            self.mask = np.packbits(bits, axis=1, bitorder="little").view(np.uint32).view(np.int32)

    def rules(self, w12):
        return w12.LogitRules(hist=i32(self.hist), hist_len=i32(self.hist_len), prompt_len=i32(self.prompt_len),
                              **{{"rep": "repetition", "freq": "frequency", "pres": "presence"}[k]: f32(v)
                                 for k, v in self.pen.items()},
                              bias=None if self.bias is None else (i32(self.bias[0]), i32(self.bias[1]), f32(self.bias[2])),
                              mask=None if self.allowed is None else i32(self.mask))

    def tree(self):
        return i32(np.concatenate(self.parents)), i32(self.draft), i32(self.off)

    def processed(self, kind=np.float32, tree=True):
        """The formula, each operation in `kind`."""
        x = self.logits.astype(kind)
        inside = lambda a: a[(a >= 0) & (a < self.V)]
        with np.errstate(all="ignore"):
            for r in range(len(self.counts)):
                h = self.hist[r, :max(0, self.hist_len[r])]
                prompt = np.bincount(inside(h[:self.prompt_len[r]]), minlength=self.V)
                said = np.bincount(inside(h[self.prompt_len[r]:]), minlength=self.V)
                bias = {}
                if self.bias is not None:
                    for j in range(self.bias[0][r], self.bias[0][r + 1]):
                        bias[int(self.bias[1][j])] = self.bias[2][j]
                for i in range(self.counts[r]):
                    m, n, p = self.off[r] + i, said.copy(), i
                    while tree and p >= 0:
                        t = self.draft[self.off[r] + p]
                        if 0 <= t < self.V:
                            n[t] += 1
                        p = self.parents[r][p]
                    if "rep" in self.pen:
                        w = kind(self.pen["rep"][r])
                        x[m] = np.where((n + prompt) > 0, np.where(x[m] > 0, x[m] / w, x[m] * w), x[m])
                    if "freq" in self.pen:
                        x[m] = np.where(n > 0, x[m] - kind(self.pen["freq"][r]) * n.astype(kind), x[m])
                    if "pres" in self.pen:
                        x[m] = np.where(n > 0, x[m] - kind(self.pen["pres"][r]), x[m])
                    for t, b in bias.items():
                        if 0 <= t < self.V:
                            x[m, t] = x[m, t] + kind(b)
            if self.allowed is not None:
                x[~self.allowed] = -np.inf
        return x

    def tokens(self):
        x = self.processed()
        tok = []
        for m in range(len(x)):
            may = np.ones(self.V, bool) if self.allowed is None else self.allowed[m]
            y = np.where(np.isnan(x[m]), -np.inf, x[m])
            best = -1
            for rank in (may & ~np.isnan(x[m]), may):    # NaN below every number
                if rank.any():
                    best = int(np.flatnonzero(rank & (y == y[rank].max()))[0])
                    break
            tok.append(best)
        return np.array(tok, np.int32)

    def check(self, out):
        got, want = out.cpu().numpy(), self.processed()
        assert np.array_equal(got, want, equal_nan=True)
        wide = self.processed(np.float64)
        fin = np.isfinite(wide)
        assert np.array_equal(np.isneginf(got), np.isneginf(wide))
        scale = np.abs(self.logits).astype(np.float64) * 1.5 + 40
        assert (np.abs(got[fin] - wide[fin]) <= 2.0 ** -21 * scale[fin]).all()

    def check_verify(self, res):
        tok, path_len, path_nodes, bonus, st = (t.cpu().numpy() for t in res)
        want = self.tokens()
        assert np.array_equal(tok, want)
        for r, n in enumerate(self.counts):
            o = self.off[r]
            if not n:
                assert path_len[r] == -1 and bonus[r] == -1
                continue
            L, path, b = oracle.accept(want[o:o + n], np.asarray(self.parents[r], np.int32), self.draft[o:o + n])
            assert path_len[r] == L and bonus[r] == b
            assert path_nodes[o:o + n].tolist() == list(path[:L + 1]) + [-1] * (n - L - 1)
        return st

    def follow(self):
        """Half the drafts repeat their parent's token under the rules, so that paths are taken
        (a changed draft changes the counts below it, so the tokens are taken as they come)."""
        rng = np.random.default_rng(1)
        for r, n in enumerate(self.counts):
            for i in range(1, n):
                if rng.random() < 0.6:
                    self.draft[self.off[r] + i] = max(0, self.tokens()[self.off[r] + self.parents[r][i]])


@pytest.mark.parametrize("V", [1, 31, 32, 33, 1000, 1024, 4095, 4097, 32001])
@pytest.mark.parametrize("counts", [[1], [16], [3, 1, 9, 2]])
def test_all_rules(w12, V, counts):
    p = Problem(V, counts, V)
    out, st = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    p.check(out)
    assert int(st) == 0


@pytest.mark.parametrize("penalties", [(), ("rep",), ("freq",), ("pres",), ("freq", "pres")])
@pytest.mark.parametrize("bias,mask", [(0, None), (7, None), (0, "half"), (300, "thin")])
def test_rules_one_by_one(w12, penalties, bias, mask):
    p = Problem(5, [4, 7], 5000, penalties=penalties, bias=bias, mask=mask)
    out, st = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    p.check(out)
    res = w12.logits_verify(f32(p.logits), p.rules(w12), *p.tree())
    p.check_verify(res)


def test_no_rules_copy_the_logits(w12):
    x = torch.randn((3, 1001), device="cuda")
    out, _ = w12.logits_process(x, w12.LogitRules(), None, None)
    assert torch.equal(out, x)


def test_rows_without_trees(w12):
    p = Problem(6, [1, 1, 1], 3001)
    out, _ = w12.logits_process(f32(p.logits), p.rules(w12), req_offsets=i32(p.off))
    assert np.array_equal(out.cpu().numpy(), p.processed(tree=False), equal_nan=True)


def test_in_place_and_strided_rows(w12):
    p = Problem(7, [5, 6], 2001)
    wide = torch.zeros((11, 2100), device="cuda")
    wide[:, 3:2004] = f32(p.logits)
    rows = wide[:, 3:2004]
    out, _ = w12.logits_process(rows, p.rules(w12), *p.tree(), out=rows)
    p.check(rows)
    assert not wide[:, :3].any() and not wide[:, 2004:].any()


def test_a_wider_mask(w12):
    p = Problem(8, [4], 1000, words=40)
    out, _ = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    p.check(out)


@pytest.mark.parametrize("hist", [1, 500, 20000])
def test_histories(w12, hist):
    p = Problem(9, [3, 2], 6000, hist=hist)
    p.hist_len[:] = [hist, hist // 2]
    p.prompt_len[:] = [hist // 3, hist // 2]              # a request with a prompt only
    out, _ = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    p.check(out)


def test_infinities_and_nan(w12):
    """In rows, in masked places and as a bias; an allowed -inf still beats a masked token."""
    p = Problem(10, [6, 4], 3000, bias=40)
    rng = np.random.default_rng(2)
    for value in (np.inf, -np.inf, np.nan, -3.4e38):
        p.logits[rng.integers(0, 10, 200), rng.integers(0, 3000, 200)] = value
    p.bias[2][:3] = -np.inf
    out, _ = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    assert np.array_equal(out.cpu().numpy(), p.processed(), equal_nan=True)
    p.check_verify(w12.logits_verify(f32(p.logits), p.rules(w12), *p.tree()))
    p = Problem(11, [2], 300, mask="half")
    p.logits[0, p.allowed[0]] = -np.inf                   # allowed but impossible
    p.logits[1, p.allowed[1]] = np.nan                    # allowed and undefined
    p.check_verify(w12.logits_verify(f32(p.logits), p.rules(w12), *p.tree()))


def test_rows_whose_mask_leaves_nothing(w12):
    p = Problem(12, [5, 3], 2500, mask="none")
    out, _ = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    assert torch.isneginf(out).all()
    tok, path_len, path_nodes, bonus, _ = w12.logits_verify(f32(p.logits), p.rules(w12), *p.tree())
    assert (tok == -1).all() and path_len.tolist() == [0, 0] and bonus.tolist() == [-1, -1]
    draft = i32(np.full(8, -1))                           # a draft of -1 does not match either
    _, path_len, _, _, _ = w12.logits_verify(f32(p.logits), p.rules(w12), p.tree()[0], draft, p.tree()[2])
    assert path_len.tolist() == [0, 0]


def test_ties_go_to_the_lowest_token(w12):
    p = Problem(13, [4], 9000, penalties=(), bias=0)
    p.logits[:] = np.round(p.logits)                      # hundreds of equal maxima
    p.check_verify(w12.logits_verify(f32(p.logits), p.rules(w12), *p.tree()))
    p.logits[:] = 0.0
    p.logits[:, ::2] = -0.0
    p.check_verify(w12.logits_verify(f32(p.logits), p.rules(w12), *p.tree()))


def test_tokens_outside_the_vocabulary_are_ignored(w12):
    p = Problem(14, [4, 4], 2000)
    p.hist[:, ::3] = -1
    p.hist[:, 1::5] = 2000
    p.hist[0, 2] = 2 ** 31 - 1
    p.draft[2], p.draft[5] = -1, 2000
    p.bias[1][1] = 2000
    p.bias[1][2] = -2 ** 31
    out, st = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    p.check(out)
    assert int(st) == 0


def test_the_last_bias_of_a_token_counts(w12):
    p = Problem(15, [3], 100, bias=300)
    out, _ = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    p.check(out)


@pytest.mark.parametrize("counts,V", [([1], 50), ([16], 20000), ([192], 3000), ([8] * 24, 4100), ([1024], 300),
                                      ([0, 5, 0, 3], 1500)])
def test_verify(w12, counts, V):
    p = Problem(16, counts, V)
    if sum(counts) <= 40:
        p.follow()
    st = p.check_verify(w12.logits_verify(f32(p.logits), p.rules(w12), *p.tree()))
    assert int(st[0]) == 0


def test_verify_agrees_with_the_two_calls(w12):
    p = Problem(17, [16, 16, 3], 30001, mask="thin")
    p.follow()
    x, rules, (parent, draft, off) = f32(p.logits), p.rules(w12), p.tree()
    out, _ = w12.logits_process(x, rules, parent, draft, off)
    a = w12.tree_verify(out, parent, draft, off)
    tok, path_len, path_nodes, bonus, _ = w12.logits_verify(x, rules, parent, draft, off)
    assert torch.equal(a[0], path_len) and torch.equal(a[2], bonus) and int(path_len.max()) > 0
    for r in range(3):
        o, n = int(off[r]), int(path_len[r]) + 1
        assert torch.equal(a[1][o:o + n], path_nodes[o:o + n])


def test_out_of_range_requests_are_reported(w12):
    for change in ("root", "child", "offsets", "nodes"):
        counts = [4, 1030 if change == "nodes" else 5, 3]
        p = Problem(18, counts, 700)
        parent, draft, off = p.tree()
        if change == "root":
            parent[4] = 0
        if change == "child":
            parent[6] = 2
        if change == "offsets":
            off = i32([0, 4, 2, 5])
        x = f32(p.logits)
        out = torch.full_like(x, 7.0)
        _, st = w12.logits_process(x, p.rules(w12), parent, draft, off, out=out)
        assert int(st) == 1
        want = p.processed()
        assert np.array_equal(out.cpu().numpy()[:4], want[:4])
        if change != "offsets":
            assert (out[4:p.off[2]] == 7.0).all()
            assert np.array_equal(out.cpu().numpy()[p.off[2]:], want[p.off[2]:])
        _, path_len, _, bonus, st = w12.logits_verify(x, p.rules(w12), parent, draft, off)
        assert int(st) == 1 and int(path_len[1]) == -1 and int(bonus[1]) == -1 and int(path_len[0]) >= 0


def test_lengths_out_of_range_are_clamped_and_reported(w12):
    p = Problem(19, [2, 2], 700)
    for at, value in (("hist_len", 10 ** 6), ("hist_len", -4), ("prompt_len", -1), ("prompt_len", 10 ** 6)):
        q = Problem(19, [2, 2], 700)
        getattr(q, at)[1] = value
        _, st = w12.logits_process(f32(q.logits), q.rules(w12), *q.tree())
        assert int(st) == 2, (at, value)
    q = Problem(19, [2, 2], 700)
    q.bias[0][2] += 50
    _, st = w12.logits_process(f32(q.logits), q.rules(w12), *q.tree())
    assert int(st) == 2
    _, st = w12.logits_process(f32(p.logits), p.rules(w12), *p.tree())
    assert int(st) == 0


def test_rows_past_32_bits(w12):
    """The last rows of logits of more than 2^31 elements."""
    M, V = 15000, 150000
    x = torch.empty((M, V), device="cuda")
    assert x.numel() > 1 << 31
    p = Problem(20, [2], V, mask=None)
    x[-2:] = f32(p.logits)
    off = i32(np.concatenate([np.arange(0, M - 2, 2), [M - 2, M]]))
    R = off.numel() - 1
    rules = w12.LogitRules(frequency=torch.full((R,), 0.25, device="cuda"))
    parent = i32(np.tile([-1, 0], M // 2))
    draft = i32(np.zeros(M))
    x[-1, 0] = 40.0
    tok, _, _, _, st = w12.logits_verify(x, rules, parent, draft, off)
    assert int(st) == 0 and int(tok[-1]) == 0
    assert int(tok[-2]) == int(x[-2].argmax())


def test_another_stream(w12):
    p = Problem(21, [16], 20000)
    s = torch.cuda.Stream()
    x, rules, t = f32(p.logits), p.rules(w12), p.tree()
    s.wait_stream(torch.cuda.current_stream())
    res = w12.logits_verify(x, rules, *t, stream=s)
    s.synchronize()
    p.check_verify(res)


def test_a_refusal_leaves_the_rules_as_they_were(w12):
    p = Problem(22, [2, 2], 700)
    x, rules, (parent, draft, off) = f32(p.logits), p.rules(w12), p.tree()
    for _ in range(2):  # the same mistake again is refused again
        with pytest.raises(ValueError, match="2 requests"):
            w12.logits_verify(x, rules, parent, draft, None)
    p.check_verify(w12.logits_verify(x, rules, parent, draft, off))


def test_out_in_place_apart_or_beside(w12):
    p = Problem(22, [2, 2], 700)
    rules, (parent, draft, off) = p.rules(w12), p.tree()
    want, st = w12.logits_process(f32(p.logits), rules, parent, draft, off)
    assert int(st) == 0
    wide = torch.zeros((5, 1500), dtype=torch.float32, device="cuda")
    x = wide[:4, :700]
    for out in (wide[1:, :700], wide[:4, 1:701], wide[:4, 699:1399], wide.as_strided((4, 700), (1500, 1), 900), wide.view(-1)[:4 * 900].view(4, 900)[:, :700]):
        with pytest.raises(w12.W12Error, match="overlap") as e:
            w12.logits_process(x, rules, parent, draft, off, out=out)
        assert e.value.status == 1
    for out in (wide[:4, 700:1400], wide[:4, 800:], wide[1:, 800:], x):
        x.copy_(f32(p.logits))
        got, st = w12.logits_process(x, rules, parent, draft, off, out=out)
        assert int(st) == 0 and torch.equal(got, want)


def test_refusals(w12):
    p = Problem(22, [2, 2], 700)
    x, rules, (parent, draft, off) = f32(p.logits), p.rules(w12), p.tree()
    with pytest.raises(ValueError):
        w12.logits_process(x.double(), rules, parent, draft, off)
    with pytest.raises(ValueError):
        w12.logits_process(x, rules, parent[:3], draft, off)
    with pytest.raises(ValueError):
        w12.logits_process(x, rules, parent, draft, None)     # rules of two requests
    with pytest.raises(ValueError):
        w12.logits_process(x[:3], rules, parent[:3], draft[:3], off)
    with pytest.raises(ValueError):
        w12.logits_process(x, rules, parent, draft, off, out=x[:, :600])
    with pytest.raises(w12.W12Error) as e:
        w12.logits_process(x, rules, parent, None, off)
    assert e.value.status == 1
    with pytest.raises(w12.W12Error) as e:
        w12.logits_verify(x, rules, None, None, off)
    assert e.value.status == 1
    with pytest.raises(w12.W12Error) as e:
        w12.logits_process(x[:1].expand(4, 700), rules, parent, draft, off)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        w12.LogitRules(hist=i32([[1, 2]]))
    with pytest.raises(ValueError):
        w12.LogitRules(repetition=f32([1.0]), presence=f32([1.0, 2.0]))


@pytest.mark.parametrize("n", [1, 2, 60])
@pytest.mark.parametrize("V", [40, 9000])
def test_a_root_that_ends_the_prompt_is_no_output(w12, n, V):
    """A request's first step: the root is its prompt's last token (prompt_len = hist_len + 1), of which
    nothing has been generated.  The root's row is then that of a call without a tree on the whole
    prompt; below the root, only drafted tokens count."""
    rng = np.random.default_rng(n * V)
    prompt = rng.integers(0, min(V, 7), n).astype(np.int32)       # tokens repeat
    draft = np.concatenate([prompt[-1:], [prompt[-1], prompt[0], 3, prompt[-1]]]).astype(np.int32)
    parent = [-1, 0, 0, 1, 3]
    x = (rng.standard_normal((5, V)) * 3).astype(np.float32)
    x[:, :7] += 30.0                                              # the prompt's tokens are the best
    rep, freq, pres = np.float32(1.3), np.float32(4.0), np.float32(8.0)
    pen = dict(repetition=f32([rep]), frequency=f32([freq]), presence=f32([pres]))
    hist = i32(np.concatenate([prompt, [0]])[None])
    first = w12.LogitRules(hist=hist, hist_len=i32([n - 1]), prompt_len=i32([n]), **pen)
    whole = w12.LogitRules(hist=hist, hist_len=i32([n]), prompt_len=i32([n]), **pen)
    want = np.empty_like(x)
    for m in range(5):
        seen, count, p = np.isin(np.arange(V), prompt), np.zeros(V, np.float32), m
        while p > 0:
            count[draft[p]] += 1
            p = parent[p]
        seen |= count > 0
        y = np.where(seen, np.where(x[m] > 0, x[m] / rep, x[m] * rep), x[m])
        y = np.where(count > 0, y - freq * count, y)
        want[m] = np.where(count > 0, y - pres, y)
    out, st = w12.logits_process(f32(x), first, i32(parent), i32(draft))
    assert int(st) == 0
    alone, _ = w12.logits_process(f32(x[:1]), whole)
    assert torch.equal(out[:1], alone)
    assert np.array_equal(out.cpu().numpy(), want)
    tok, path_len, _, bonus, st = w12.logits_verify(f32(x), first, i32(parent), i32(draft))
    assert int(st) == 0 and tok.tolist() == want.argmax(1).tolist()
    length, _, last = oracle.accept(want.argmax(1).astype(np.int32), np.asarray(parent, np.int32), draft)
    assert int(path_len) == length and int(bonus) == last


def test_a_prompt_ends_at_the_root(w12):
    """One token more than the history and the root is out of range, as is one more than the history without a tree."""
    hist, x = i32([[1, 2, 3, 4]]), torch.zeros((1, 50), device="cuda")
    for prompt, tree, want in ((4, True, 0), (5, True, 2), (3, False, 0), (4, False, 2)):
        rules = w12.LogitRules(hist=hist, hist_len=i32([3]), prompt_len=i32([prompt]), frequency=f32([1.0]))
        _, st = w12.logits_process(x, rules, *([i32([-1]), i32([4])] if tree else []))
        assert int(st) == want, (prompt, tree)


@pytest.mark.parametrize("n", range(1, 13))
def test_a_history_that_ends_with_its_array(w12, n):
    """The last row's history may be the array's last entries: nothing behind hist_len is needed."""
    V, stride = 300, 12
    rng = np.random.default_rng(n)
    hist = i32(rng.integers(0, 9, stride + n))
    hist_len, freq, off = i32([stride, n]), f32([0.5, 0.25]), i32([0, 1, 2])
    x = torch.randn((2, V), device="cuda")
    out, st = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    r = w12.logit_rules()
    r.hist, r.hist_stride, r.hist_len, r.freq = hist.data_ptr(), stride, hist_len.data_ptr(), freq.data_ptr()
    assert w12.lib().logits_process(x.data_ptr(), V, 2, V, ctypes.byref(r), None, None, off.data_ptr(), 2, out.data_ptr(), V,
                                    st.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    count = torch.stack([torch.bincount(hist[:stride], minlength=V), torch.bincount(hist[stride:], minlength=V)])
    assert torch.equal(out, x - freq[:, None] * count) and int(st) == 0
