"""tree_verify_sampled against the definition in 64 bits, step by step as the header states it: rows of
probabilities, renormalised after every refusal.  Paths and tokens are whole numbers and have to be equal; the
seeds are fixed, and a number falls within 2^-28 of a border once in millions of draws."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

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


def target(l, T):
    """The target's probabilities (not normalised) of a row; none: zeros."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    if T < 1e-5:
        p = np.zeros_like(l)
        p[np.argmax(l)] = 1.0
        return p
    if top == np.inf:
        return (l == np.inf).astype(np.float64)
    return np.exp((l - top) / T)


def one_request(logits, probs, T, parent, draft, u, u_bonus):
    """path, bonus"""
    V, n = logits.shape[1], len(parent)
    clamp = lambda x: min(max(float(np.nan_to_num(x, nan=0.0)), 0.0), float(np.float32(0.99999994)))
    cur, path = 0, [0]
    while True:
        p = target(logits[cur], T)
        has = p.sum() > 0
        p = p / p.sum() if has else p
        start = p
        q = None if probs is None else np.clip(np.nan_to_num(probs[cur].astype(np.float64), nan=0.0), 0.0, 1.0)
        Q, spent, seen, taken = 1.0, False, set(), None
        for c in range(1, n):
            if parent[c] != cur:
                continue
            x = int(draft[c])
            if not 0 <= x < V or not has or spent or x in seen:
                continue
            seen.add(x)
            if probs is not None and Q <= 0:
                continue
            qx = 1.0 if q is None else q[x] / Q
            if clamp(u[c]) * qx < p[x]:
                taken = c
                break
            if q is None:
                left = p.copy()
                left[x] = 0.0
            else:
                if q[x] == 0:
                    continue
                left = np.maximum(p - q / Q, 0.0)
                Q -= q[x]
                q = q.copy()
                q[x] = 0.0
            if left.sum() > 0:
                p = left / left.sum()
            else:
                p = start
                spent = q is not None
                if q is None:
                    p, spent = start, True
        if taken is None:
            if not has:
                return path, -1
            cum = np.cumsum(p)
            over = np.nonzero((cum > clamp(u_bonus) * cum[-1]) & (p > 0))[0]
            return path, int(over[0] if len(over) else np.nonzero(p > 0)[0][-1])
        cur = taken
        path.append(taken)


class Problem:
    def __init__(self, seed, counts, V, probs=True, temperature="mixed", sd=3.0, shape="tree", good=0.8):
        rng = np.random.default_rng(seed)
        self.counts, self.V = counts, V
        R, M = len(counts), sum(counts)
        self.off = np.concatenate([[0], np.cumsum(counts)])
        up = {"tree": lambda i: int(rng.integers(max(0, i - 4), i)), "chain": lambda i: i - 1, "star": lambda i: 0}[shape]
        self.parent = [[-1] + [up(i) for i in range(1, n)] if n else [] for n in counts]
        self.logits = (rng.standard_normal((M, V)) * sd).astype(np.float32)
        for m in range(M):
            self.logits[m, rng.integers(0, V, 3)] += rng.uniform(3, 9, 3).astype(np.float32)
        self.T = None
        if temperature == "mixed":
            self.T = rng.uniform(0.5, 1.5, R).astype(np.float32)
            self.T[rng.random(R) < 0.2] = 0.0
        guess = self.logits * 0.9 + rng.standard_normal((M, V)) * (1 - good) * sd
        guess = np.exp(guess - guess.max(1, keepdims=True))
        guess /= guess.sum(1, keepdims=True)
        self.probs = guess.astype(np.float32) if probs else None
        self.draft = np.zeros(M, np.int32)
        key = np.log(guess + 1e-30) + (rng.gumbel(size=(M, V)) if probs else 0)
        for r, par in enumerate(self.parent):
            kids = {}
            for i in range(1, len(par)):
                k = kids[par[i]] = kids.get(par[i], -1) + 1
                row = self.off[r] + par[i]
                order = np.argpartition(-key[row], min(k, V - 1))[:k + 1]
                self.draft[self.off[r] + i] = order[np.argsort(-key[row][order])][min(k, V - 1)]
        self.u, self.ub = rng.random(M).astype(np.float32), rng.random(R).astype(np.float32)

    def want(self):
        path, length, bonus = np.full(sum(self.counts), -1, np.int32), [], []
        for r, n in enumerate(self.counts):
            if n == 0:
                length.append(-1)
                bonus.append(-1)
                continue
            s = slice(self.off[r], self.off[r + 1])
            p, b = one_request(self.logits[s], None if self.probs is None else self.probs[s],
                               1.0 if self.T is None else self.T[r], self.parent[r], self.draft[s], self.u[s], self.ub[r])
            path[self.off[r]:self.off[r] + len(p)] = p
            length.append(len(p) - 1)
            bonus.append(b)
        return length, path.tolist(), bonus

    def args(self):
        return dict(parent=i32(np.concatenate([np.asarray(p, np.int32) for p in self.parent])), draft=i32(self.draft), u=f32(self.u),
                    u_bonus=f32(self.ub), temperature=None if self.T is None else f32(self.T), req_offsets=i32(self.off))

    def check(self, w12, logits=None, probs=None, **kw):
        logits = f32(self.logits) if logits is None else logits
        if self.probs is not None and probs is None:
            probs = f32(self.probs)
        length, path, bonus, status = w12.tree_verify_sampled(logits, draft_probs=probs, **self.args(), **kw)
        assert int(status) == 0
        got = length.tolist(), path.tolist(), bonus.tolist()
        assert got == self.want()
        return got


SHAPES = [([1], 7), ([8], 33), ([16], 1000), ([5, 0, 1, 12], 1023), ([8] * 24, 1025), ([3, 2] * 40, 130), ([64], 4099),
          ([6] * 3, 32000), ([2, 7], 50257), ([9], 151936), ([1] * 5, 151936), ([3, 1], 300007),
          ([1, 2, 3], 1), ([4, 4], 2)]


@pytest.mark.parametrize("counts,V", SHAPES)
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("temperature", [None, "mixed"])
def test_trees(w12, counts, V, probs, temperature):
    for seed in range(3):
        Problem(seed + V, counts, V, probs, temperature).check(w12)


@pytest.mark.parametrize("shape,counts,V", [("chain", [60], 500), ("chain", [5] * 64, 300), ("star", [100], 700),
                                            ("star", [30] * 4, 9000), ("star", [9], 4)])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("good", [0.3, 1.0])
def test_chains_and_stars(w12, shape, counts, V, probs, good):
    for seed in range(3):
        Problem(seed, counts, V, probs, "mixed", sd=1.0, shape=shape, good=good if V > 4 else 0.3).check(w12)


@pytest.mark.parametrize("n", [1024])
def test_largest_tree(w12, n):
    Problem(1, [n], 67, True, "mixed", sd=1.0).check(w12)
    Problem(1, [n], 67, False, "mixed", sd=1.0, shape="chain").check(w12)


@pytest.mark.parametrize("V", [1, 5, 1000, 33001])
def test_strides_and_alignment(w12, V):
    p = Problem(2, [7, 5], V)
    for pad, shift, other in ((1, 0, 0), (8, 1, 1), (4, 4, 2), (4 - V % 4, 0, 3), (0, 0, 0), (0, 3, 1)):
        big = [torch.full((12 * (V + pad) + 8,), 50.0, device="cuda") for _ in range(2)]
        l, q = (b[s:s + 12 * (V + pad)].view(12, V + pad)[:, :V] for b, s in zip(big, (shift, other)))
        l.copy_(f32(p.logits))
        q.copy_(f32(p.probs))
        p.check(w12, logits=l, probs=q)


@pytest.mark.parametrize("V", [700, 9001])
def test_rising_and_falling_rows(w12, V):
    """Rows whose largest logit grows from one stretch of tokens to the next, and ends in a jump."""
    for seed, order in enumerate((1, -1)):
        p = Problem(seed, [1, 3, 1, 2], V, temperature=None)
        rise = np.linspace(-40.0, 30.0, V)[::order].astype(np.float32)
        p.logits = (rise + 0.1 * p.logits).astype(np.float32)
        p.logits[0, -1] = 90.0
        p.logits[4, V // 2:] = -np.inf
        p.logits[4, :V // 3] = -np.inf
        p.ub[[0, 2]] = 0.2, 0.999
        p.check(w12)


def test_masked_rows(w12):
    """-inf, NaN, the lowest float and +inf; rows with one token, rows with none."""
    for seed in range(4):
        p = Problem(seed, [8, 6, 9, 4], 500, probs=seed % 2 == 0, temperature="mixed" if seed < 2 else None)
        rng = np.random.default_rng(seed)
        p.logits[rng.random(p.logits.shape) < 0.5] = -np.inf
        p.logits[rng.random(p.logits.shape) < 0.05] = np.nan
        p.logits[rng.random(p.logits.shape) < 0.05] = np.finfo(np.float32).min
        p.logits[3, :] = -np.inf
        p.logits[3, 77] = -4.0
        p.logits[8, :] = -np.inf            # a root that allows nothing
        p.logits[14, 10:20] = np.inf
        p.logits[15, :] = np.nan
        p.logits[23, :] = np.finfo(np.float32).min
        got = p.check(w12)
        assert got[2][1] == -1


@pytest.mark.parametrize("T", [0.0, 9.9e-6, 1e-4, 0.01, 1.0, 30.0, 1e6, np.inf])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 300.0, 1e30])
def test_temperatures_and_sizes(w12, T, scale):
    p = Problem(5, [6, 5, 1], 2000, temperature=None)
    p.logits = (p.logits * np.float32(scale)).astype(np.float32)
    p.T = np.full(3, T, np.float32)
    p.check(w12)


def test_shifted_logits(w12):
    """Logits far from zero, where the largest is no multiple of the others' last place."""
    for shift in (-1000.0, -17.3, 1e4, 3e5):
        p = Problem(6, [9, 4], 3001, sd=1.0)
        p.logits = (p.logits + np.float32(shift)).astype(np.float32)
        p.check(w12)


def test_equal_tokens_and_greedy_ties(w12):
    p = Problem(7, [5, 5], 300)
    p.logits[:] = 1.25
    p.T = np.array([0.0, 1.0], np.float32)
    p.check(w12)


def test_drafts_that_cannot_be_taken(w12):
    """Outside the vocabulary, twice under one node, impossible for the drafter, and certain for it."""
    for seed in range(6):
        p = Problem(seed, [40, 12], 30, probs=seed % 2 == 0, temperature=None, sd=1.0, shape="star")
        rng = np.random.default_rng(seed)
        p.draft[rng.integers(1, 40, 6)] = [-1, 30, 2 ** 31 - 1, -2 ** 31, 31, -7]
        p.draft[20:30] = p.draft[2:12]
        if p.probs is not None:
            p.probs[0, rng.integers(0, 30, 12)] = 0.0
            p.probs[0, 3] = np.nan
            p.probs[0, 4] = -0.5
            p.probs[40] = 0.0
            p.probs[40, p.draft[42]] = 1.0     # the second child was certain: none can follow it
        p.u[:] = np.maximum(p.u, 0.9)          # many refusals
        p.check(w12)


def test_nothing_left(w12):
    """A drafter that is above the target everywhere, and children that hold all of p."""
    p = Problem(3, [4], 50, temperature=None, shape="star")
    p.probs[:] = 1.0
    p.u[:] = 0.999
    p.check(w12)
    p = Problem(3, [4], 50, probs=False, temperature=None, shape="star")
    p.logits[0] = -np.inf
    p.logits[0, p.draft[1:4]] = [1.0, 0.5, 0.0]
    p.u[:] = 0.99999994
    p.check(w12)


@pytest.mark.parametrize("counts", [[2], [4], [2, 4, 7] * 8, [2] * 64])
def test_rounds_that_end_and_go_on(w12, counts):
    """A last sum that leaves nothing is followed by another round, beside requests that end with theirs; every
    run gives the same."""
    p = Problem(13, counts, 40000, temperature=None, shape="star")
    for r in range(0, len(counts), 2):
        s = slice(p.off[r], p.off[r + 1])
        p.probs[s] = 1.0
        p.u[s] = 0.999
    got, ws = p.check(w12), w12.Workspace()
    logits, probs, a = f32(p.logits), f32(p.probs), p.args()
    runs = [w12.tree_verify_sampled(logits, draft_probs=probs, ws=ws, **a) for _ in range(50)]
    assert all(tuple(t.tolist() for t in x[:3]) == got and int(x[3]) == 0 for x in runs)


def test_numbers_at_the_ends(w12):
    for u, ub in ((0.0, 0.0), (1.0, 1.0), (np.nan, np.nan), (-3.0, 5.0), (0.99999994, 0.99999994)):
        p = Problem(4, [6, 3], 777, temperature=None)
        p.u[:] = u
        p.ub[:] = ub
        p.check(w12)


def test_requests_out_of_range(w12):
    p = Problem(8, [4, 3, 5, 2, 6], 900)
    p.T = np.array([1.0, -0.5, 0.7, np.nan, 1.0], np.float32)
    a = p.args()
    a["parent"][7] = 0                      # request 2's root
    length, path, bonus, status = w12.tree_verify_sampled(f32(p.logits), draft_probs=f32(p.probs), **a)
    assert int(status) == 1
    p.T[[1, 3]] = 1.0
    want = p.want()
    for r in range(5):
        s = slice(p.off[r], p.off[r + 1])
        if r in (1, 2, 3):
            assert (int(length[r]), int(bonus[r])) == (-1, -1) and path[s].tolist() == [-1] * p.counts[r]
        else:
            assert (int(length[r]), int(bonus[r]), path[s].tolist()) == (want[0][r], want[2][r], want[1][s])
    want = p.want()
    for off, bad in (([0, 4, 3, 12, 14, 20], range(5)), ([0, 4, 7, 12, 14, 21], [4]), ([-1, 4, 7, 12, 14, 20], [0])):
        a = p.args()
        a["req_offsets"] = i32(off)
        length, _, bonus, status = w12.tree_verify_sampled(f32(p.logits), draft_probs=f32(p.probs), **a)
        assert int(status) == 1
        for r in range(5):
            assert (int(length[r]), int(bonus[r])) == ((-1, -1) if r in bad else (want[0][r], want[2][r])), (off, r)
    one = Problem(1, [1025], 10, temperature=None)
    length, _, bonus, status = w12.tree_verify_sampled(f32(one.logits), draft_probs=f32(one.probs), **one.args())
    assert (int(length), int(bonus), int(status)) == (-1, -1, 1)


def test_far_rows(w12):
    """Rows past 2^31 elements."""
    p = Problem(9, [20], 600, temperature=None)
    big = [torch.empty(20, 1 << 27, device="cuda") for _ in range(2)]
    l, q = (b[:, :600] for b in big)
    l.copy_(f32(p.logits))
    q.copy_(f32(p.probs))
    p.check(w12, logits=l, probs=q)


def test_repeated_streams_and_graphs(w12):
    p = Problem(10, [8] * 6, 20000)
    ws = w12.Workspace()
    got = p.check(w12, ws=ws)
    for _ in range(3):
        assert p.check(w12, ws=ws) == got
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert p.check(w12, ws=ws) == got
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    logits, probs, a = f32(p.logits), f32(p.probs), p.args()
    out = [w12.tree_verify_sampled(logits, draft_probs=probs, ws=ws, stream=x, **a) for x in (s, s2, None)]
    torch.cuda.synchronize()
    for o in out:
        assert tuple(t.tolist() for t in o[:3]) == got
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = w12.tree_verify_sampled(logits, draft_probs=probs, ws=ws, **a)
    p2 = Problem(11, [8] * 6, 20000)
    logits.copy_(f32(p2.logits))
    probs.copy_(f32(p2.probs))
    for k, v in p2.args().items():
        a[k].copy_(v)
    g.replay()
    torch.cuda.synchronize()
    assert tuple(t.tolist() for t in o[:3]) == p2.want()


def test_text_is_distributed_as_the_target(w12):
    """First tokens of 60000 requests with one pair of rows, drafted by chance: counts against p.  A count's
    standard deviation is at most sqrt(n)/2 = 122; five of them bound all six tokens together to 4e-6."""
    rng = np.random.default_rng(0)
    R, V = 60000, 6
    row = np.array([1.0, 0.2, -0.5, 0.7, -1.5, 0.1], np.float32)
    q = np.array([0.05, 0.3, 0.25, 0.1, 0.2, 0.1], np.float32)
    order = np.argsort(-(np.log(q) + rng.gumbel(size=(R, V))), 1)       # draws without replacement
    T = np.float32(0.8)
    p = np.exp(row.astype(np.float64) / T)
    p /= p.sum()
    parent = np.tile([-1, 0, 0, 0], R)
    draft = np.concatenate([np.zeros((R, 1), np.int64), order[:, :3]], 1).ravel()
    for probs in (True, False):
        if not probs:
            draft = np.tile([0, 1, 3, 4], R)                            # the same children every time
        length, path, bonus, status = w12.tree_verify_sampled(
            f32(row).expand(4 * R, V).contiguous(), i32(parent), i32(draft), f32(rng.random(4 * R)), f32(rng.random(R)),
            draft_probs=f32(q).expand(4 * R, V).contiguous() if probs else None, temperature=f32(np.full(R, T)),
            req_offsets=i32(np.arange(R + 1) * 4))
        assert int(status) == 0
        first = path.view(R, 4)[:, 1].long()
        tok = torch.where(length > 0, i32(draft).view(R, 4).gather(1, first.clamp(min=0)[:, None])[:, 0], bonus)
        counts = torch.bincount(tok.long(), minlength=V).cpu().numpy()
        assert (np.abs(counts - R * p) < 5 * np.sqrt(R) / 2).all(), (counts, R * p)
