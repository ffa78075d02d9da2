"""tree_verify_sampled beside the borders of its decisions: a number just below and just above a token's
probability, and just below and above a border of the cumulative sum.

Every row has one token of small mass whose logit is set so that the border stands at a given distance of the number
(by float64 sums, good to 2^-40 here).  Distances are in units of p's sum.  What the kernel is allowed: its masses are good to
2.8e-9 of themselves (two roundings of the reduced argument by 2^-31, of which ln 2 counts, the polynomial's last two steps
and the low part's product 2^-30.5, 2^-31, 2^-30.5, what its terms leave out 2^-33, the rest of the slope 2^-32), its
sums add 2^-30.5 (the sum of two low parts), so an error is below 3.5e-9 of the sum, and at a border u of one sum it
counts u (1 - u) <= 1/4 from either side: 1.8e-9, less than 2^-28 = 3.7e-9.  Without q a refused token's mass only leaves the
sum: 2.8e-9 p + u 3.5e-9 < 3e-9 for the shares below.  With q a refusal leaves e - tau q, three roundings of
2^-30.5 more, in sums one more of that for a low part above the sum so far: 6.1e-9, and q tau adds 3.5e-9 of what
q is left (1/2): M' is off by less than 8e-9, tau by 3.5e-9.  With q = 1/4 and Q = 1/2 at a second child the decision's
error is below 2.8e-9 p + 3.5e-9 / 4 + 8e-9 / 2 < 7e-9, half of 2^-26 = 1.5e-8.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_sampled import f32, i32, one_request

pytestmark = pytest.mark.gpu
V = 151936


@pytest.fixture(scope="module")
def w12():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lossless_bit_weights_gb300 as m
    m.lib()
    return m


def tuned(margin, T, size, at, least):
    """A float32 logit of the tuning token, whose mass is about `size` times e^0: margin(its mass) (about linear) comes to
    least .. 2 least in the direction of the sign of `least`."""
    goal, a = 1.5 * least, size
    b = size * 1.01
    fa, fb = margin(a) - goal, margin(b) - goal
    for _ in range(6):
        if fa == fb:
            break
        a, b, fa = b, b - fb * (b - a) / (fb - fa), fb
        assert b > 0, "the tuning token cannot bring the border there"
        fb = margin(b) - goal
    l = np.float32(at + T * np.log(b))
    got = margin(np.exp((float(l) - at) / T))
    assert 1.0 <= got / least <= 2.0, got
    return l


def flat_rows(R, seed, side, least, q=1.0, V=V):
    """R rows of one token (0) with u q of the mass or so, one (1) that tunes it, all others equal.  Token 0's
    share (bonus: tokens 0 and 1) stands `least` above u q, or below where side is -1."""
    rng = np.random.default_rng(seed)
    T, low = rng.uniform(0.5, 1.5, R).astype(np.float32), rng.uniform(-3, 0, R).astype(np.float32)
    u = rng.uniform(0.45, 0.55, R).astype(np.float32) if q == 1.0 else rng.uniform(0.6, 0.73, R).astype(np.float32)
    head = np.zeros((R, 2), np.float32)
    for r in range(R):
        t, want = float(T[r]), float(u[r]) * q
        rest = V - 2.0                                   # masses in units of the equal ones
        if q == 1.0:
            head[r, 0] = np.float32(low[r] + t * np.log(0.998 * rest * want / (1 - want)))
            e0 = np.exp((float(head[r, 0]) - float(low[r])) / t)
            margin = lambda e: (e0 + e) / (e0 + e + rest) - want
            head[r, 1] = tuned(margin, t, 0.002 * rest, float(low[r]), side[r] * least)
        else:
            head[r, 0] = np.float32(low[r] + t * np.log(1.002 * rest * want / (1 - want)))
            e0 = np.exp((float(head[r, 0]) - float(low[r])) / t)
            margin = lambda e: e0 / (e0 + e + rest) - want
            head[r, 1] = tuned(margin, t, 0.002 * rest, float(low[r]), side[r] * least)
    return T, low, head, u


@pytest.mark.parametrize("R,V", [(1, V), (9, V), (200, V), (160, 600001)])
def test_bonus_of_flat_rows(w12, R, V):
    """Half of the mass in equal tokens, whose low parts all have one sign; with 200 requests a warp sums 9496 of them,
    with 160 of the largest rows 37632."""
    side = np.where(np.arange(R) % 2 == 0, 1, -1)
    for seed in range(8 if R < 100 else 1):
        T, low, head, u = flat_rows(R, seed, side, 2.0 ** -28, V=V)
        logits = f32(low)[:, None].expand(R, V).clone()
        logits[:, :2] = f32(head)
        none = i32(np.full(R, -1))
        length, _, bonus, status = w12.tree_verify_sampled(logits, none, i32(np.zeros(R)), f32(np.zeros(R)), f32(u),
                                                           temperature=f32(T), req_offsets=i32(np.arange(R + 1)))
        assert int(status) == 0 and length.tolist() == [0] * R
        assert bonus.tolist() == np.where(side > 0, 1, 2).tolist()


@pytest.mark.parametrize("R", [4, 512])
@pytest.mark.parametrize("probs", [True, False])
def test_acceptance_on_flat_rows(w12, R, probs):
    """The same rows with a child of token 0; with 512 of them a warp of the rows' kernel sums 21504 tokens."""
    q = 0.75 if probs else 1.0
    side = np.where(np.arange(R) % 3 == 0, 1, -1)
    if probs:
        T, low, head, u = flat_rows(R, 1, side, 2.0 ** -28, q)
    else:  # (tokens 0 and 1 change places: token 0 alone is the share)
        T, low, head, _ = flat_rows(R, 2, side, 2.0 ** -28, 0.75)
        u = np.zeros(R, np.float32)
        for r in range(R):
            t, rest, at = float(T[r]), V - 2.0, float(low[r])
            e0 = np.exp((float(head[r, 0]) - at) / t)
            u[r] = np.float32(e0 / (e0 + 0.002 * rest + rest))
            head[r, 1] = tuned(lambda e: e0 / (e0 + e + rest) - float(u[r]), t, 0.002 * rest, at, side[r] * 2.0 ** -28)
    logits = f32(low).repeat_interleave(2)[:, None].expand(2 * R, V).clone()
    logits[::2, :2] = f32(head)
    p = None
    if probs:
        p = torch.zeros((2 * R, V), device="cuda")
        p[:, 0], p[:, 5] = 0.75, 0.25
    both = np.stack([np.zeros(R), u], 1).ravel()
    length, _, _, status = w12.tree_verify_sampled(
        logits, i32(np.tile([-1, 0], R)), i32(np.zeros(2 * R)), f32(both), f32(np.full(R, 0.5)), draft_probs=p,
        temperature=f32(T), req_offsets=i32(2 * np.arange(R + 1)))
    assert int(status) == 0
    assert length.tolist() == (side > 0).tolist()


def random_row(rng, share):
    """A row's logits, temperature, and the tuning token (2^-12 of the mass); tokens of `share` have that part of it."""
    T = float(np.float32(rng.uniform(0.6, 1.3)))
    l = (rng.standard_normal(V) * 3).astype(np.float32)
    y = int(rng.integers(V // 8, V // 4))
    named = dict(share)
    named[y] = 2.0 ** -12
    idx = np.array(list(named))
    e = np.exp(l.astype(np.float64) / T)
    e[idx] = 0
    total = e.sum() / (1 - sum(named.values()))
    for v, part in named.items():
        l[v] = np.float32(T * np.log(part * total))
    return l, T, y


def masses(l, T):
    return np.exp(l.astype(np.float64) / T)


def call(w12, logits, T, draft, u, ub, probs=None):
    """Requests of one root with children each; path lengths, first nodes, bonus tokens."""
    R, n = len(T), len(draft[0])
    length, path, bonus, status = w12.tree_verify_sampled(
        f32(np.concatenate(logits)), i32(np.tile([-1] + [0] * (n - 1), R)), i32(np.concatenate(draft)), f32(np.concatenate(u)),
        f32(ub), draft_probs=None if probs is None else f32(np.concatenate(probs)), temperature=f32(T),
        req_offsets=i32(n * np.arange(R + 1)))
    assert int(status) == 0
    return length.tolist(), path.view(R, n).tolist(), bonus.tolist()


@pytest.mark.parametrize("R", [1, 8])
def test_bonus_of_random_rows(w12, R):
    for seed in range(4):
        rng = np.random.default_rng(seed + 100 * R)
        rows, Ts, ubs, want = [], [], [], []
        for r in range(R):
            l, T, y = random_row(rng, {})
            e = masses(l, T)
            k = int(rng.integers(V // 4, V - 1000))
            while min(e[k], e[k + 1]) < 2.0 ** -22 * e.sum():
                k += 1
            u = float(np.float32(e[:k + 1].sum() / e.sum()))
            side = 1 if r % 2 == 0 else -1
            e[y] = 0
            before, after = e[:k + 1].sum(), e[k + 1:].sum()
            l[y] = tuned(lambda m: (before + m) / (before + m + after) - u, T, 2.0 ** -12 * (before + after), 0.0,
                         side * 2.0 ** -28)
            path, token = one_request(l[None], None, T, [-1], [0], [0.0], u)
            assert token == (k if side > 0 else k + 1)
            rows.append(l[None])
            Ts.append(T)
            ubs.append(u)
            want.append(token)
        zero = [np.zeros(1)] * R
        assert call(w12, rows, Ts, zero, zero, ubs)[2] == want


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("R", [1, 8])
def test_first_child_on_random_rows(w12, R, probs):
    for seed in range(4):
        rng = np.random.default_rng(seed + 10 * R + probs)
        rows, Ts, drafts, us, qs, ubs, want = [], [], [], [], [], [], []
        for r in range(R):
            x, other = (int(v) for v in rng.choice(V // 8, 2, replace=False))
            l, T, y = random_row(rng, {x: rng.uniform(0.1, 0.6)})
            q = 0.75 if probs else 1.0
            e = masses(l, T)
            u = float(np.float32(e[x] / e.sum() / q))
            e[y] = 0
            side = 1 if r % 2 == seed % 2 else -1
            rest = e.sum()
            l[y] = tuned(lambda m: e[x] / (rest + m) - u * q, T, 2.0 ** -12 * rest, 0.0, side * 2.0 ** -28)
            p = np.zeros((2, V), np.float32)
            p[:, x], p[:, other] = 0.75, 0.25
            row = np.stack([l, (rng.standard_normal(V) * 3).astype(np.float32)])
            path, token = one_request(row, p if probs else None, T, [-1, 0], [0, x], [0.0, u], 0.37)
            assert len(path) == (2 if side > 0 else 1)
            rows.append(row)
            Ts.append(T)
            drafts.append(np.array([0, x]))
            us.append(np.array([0.0, u]))
            qs.append(p)
            ubs.append(0.37)
            want.append((len(path) - 1, token))
        length, _, bonus = call(w12, rows, Ts, drafts, us, ubs, qs if probs else None)
        assert list(zip(length, bonus)) == want


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("R", [1, 8])
def test_second_child_on_random_rows(w12, R, probs):
    """The border of a second child once the first is refused.  Without q that is u (1 - p(first)) of the first sum."""
    least = 2.0 ** -26 if probs else 2.0 ** -28
    for seed in range(4):
        rng = np.random.default_rng(seed + 10 * R + probs)
        rows, Ts, drafts, us, qs, ubs, want = [], [], [], [], [], [], []
        for r in range(R):
            a, b, other = (int(v) for v in rng.choice(V // 8, 3, replace=False))
            l, T, y = random_row(rng, {a: rng.uniform(0.2, 0.3), b: rng.uniform(0.3, 0.36)})
            e = masses(l, T)
            p = rng.random(V).astype(np.float32) * (e < np.median(e))  # (the drafter likes what the target does not)
            p[[a, b, y]] = 0
            p *= np.float32(0.25) / p.sum()
            p[a], p[b] = 0.5, 0.25
            p64 = p.astype(np.float64)
            e[y] = 0

            def share(m):
                """What the first refusal leaves of b, over its sum; and that sum over the first one."""
                f = e.copy()
                f[y] = m
                f /= f.sum()
                left = np.maximum(f - p64, 0) if probs else np.where(np.arange(V) == a, 0, f)
                return left[b] / left.sum(), left.sum()

            size = 2.0 ** -12 * e.sum()
            u = float(np.float32(share(size)[0] * (2 if probs else 1)))
            assert 0.05 < u < 0.95
            side = 1 if r % 2 == seed % 2 else -1

            def margin(m):
                s, left = share(m)
                return (s - u * (0.5 if probs else 1)) * left

            l[y] = tuned(margin, T, size, 0.0, side * least)
            row = np.stack([l, *(rng.standard_normal((2, V)) * 3).astype(np.float32)])
            p = np.stack([p] * 3)
            path, token = one_request(row, p if probs else None, T, [-1, 0, 0], [0, a, b], [0.0, 0.9, u], 0.61)
            assert path == ([0, 2] if side > 0 else [0])
            rows.append(row)
            Ts.append(T)
            drafts.append(np.array([0, a, b]))
            us.append(np.array([0.0, 0.9, u]))
            qs.append(p)
            ubs.append(0.61)
            want.append((len(path) - 1, token))
        length, _, bonus = call(w12, rows, Ts, drafts, us, ubs, qs if probs else None)
        assert list(zip(length, bonus)) == want


@pytest.mark.parametrize("a,side", [(-1.3634447, 1), (-0.06020798, -1)])
def test_rough_sum_of_a_long_row(w12, a, side):
    """A row of 2^31 tokens without q, whose decision a rough sum must not take: tokens of mass 1 and e^a, e^a, e^a in turn,
    so that a lane's additions of 1 + 3 e^a all round one way (4600 of them lose 6.8e-5 of the sum; sums tell apart what is
    6.2e-5 away).  The number stands 2e-6 of itself from p."""
    n, x = (1 << 31) - (1 << 14), (1 << 31) - (1 << 15)
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 40 GB")
    logits = torch.zeros((2, n), device="cuda")
    logits[0].view(-1, 4)[:, 1:] = a
    logits[0, x] = 16.0
    e = np.exp(float(np.float32(a)))
    p = np.exp(16.0) / (n / 4 * (1 + 3 * e) - 1 + np.exp(16.0))
    u = np.float32(p * (1 - side * 2e-6))
    length, path, _, status = w12.tree_verify_sampled(logits, i32([-1, 0]), i32([0, x]), f32([0.0, u]), f32([0.5]))
    assert int(status) == 0 and length.tolist() == [side > 0] and path.tolist() == ([0, 1] if side > 0 else [0, -1])


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("probs", [None, True, False])
def test_borders_between_far_logits(w12, rising, probs):
    """Logits whose exponents pass 2^16, two tokens a row in ranges of their own: parts of a row then differ by no power of two.
    Without drafts (probs None) the bonus' border, else the child's.  All but that factor is exact here, and that is a
    pair of floats, so 2^-28 is far from what may come out."""
    R, V = 256, 4100
    a, b = (3000, 200) if rising else (200, 3000)         # the larger logit's token, and the other
    rng = np.random.default_rng(7)
    q, rows, T, u, want = 0.875 if probs else 1.0, np.full((R, V), -np.inf, np.float32), [], [], []
    while len(u) < R:
        t = float(np.float32(rng.uniform(0.8, 1.2)))
        d = 0.03125 * int(rng.integers(1, 50))
        p = 1 / (1 + np.exp(-d / t))                       # of a
        first = p if a < b or probs is not None else 1 - p  # the border: of the lower token, or of the child's
        n = np.float32(first / q)
        for x in (n, np.nextafter(n, np.float32(0)), np.nextafter(n, np.float32(1))):
            gap = float(x) * q - first
            if 2.0 ** -28 < abs(gap) < 2.0 ** -26 and x < 1 and len(u) < R:
                rows[len(u), a], rows[len(u), b] = 2.0 ** 18, 2.0 ** 18 - d
                T.append(t)
                u.append(x)
                want.append(gap < 0)
    want = np.array(want)
    assert 50 < want.sum() < R - 50
    zero, off = np.zeros(R), np.arange(R + 1)
    if probs is None:
        length, _, bonus, status = w12.tree_verify_sampled(f32(rows), i32(zero - 1), i32(zero), f32(zero), f32(u),
                                                           temperature=f32(T), req_offsets=i32(off))
        assert int(status) == 0 and (bonus.cpu().numpy() == np.where(want, min(a, b), max(a, b))).all()
        return
    pr = np.zeros(V, np.float32)
    pr[a], pr[7] = q, 1 - q
    length, _, _, status = w12.tree_verify_sampled(
        f32(np.repeat(rows, 2, 0)), i32(np.tile([-1, 0], R)), i32(np.tile([0, a], R)), f32(np.stack([zero, u], 1).ravel()),
        f32(zero), draft_probs=f32(np.tile(pr, (2 * R, 1))) if probs else None, temperature=f32(T), req_offsets=i32(2 * off))
    assert int(status) == 0 and (length.cpu().numpy() == want).all()
