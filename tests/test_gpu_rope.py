"""tree_positions, qkv_rope and kv_append against the formulas in 64 bits.

Tolerance of q, k and v: one rounding to bf16 (half a step, 2^-8 of the value), and the float arithmetic before
it.  There the norm's factor is off by less than 2^-19 (a float sum of at most 256 squares in a tree of depth 8 behind 8
serial ones: 16 roundings; rsqrt two steps, three products), sine and cosine by 2^-22 of one (their
own two steps and the angle's rounding to 2^-25 turns, 1.9e-7), the pair's two products and sum by
3 * 2^-24: less than 2^-18 of the two columns' sizes together.
"""
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


class Rows:
    """A projection's rows with a form, and q, k, v by the formula in 64 bits."""

    def __init__(self, w12, seed, M, hq, hkv, d, rot, norm="qk", interleaved=False, kind="float", pos_hi=5000, scale=1.0,
                 stride=0, eps=1e-6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = (hq + 2 * hkv) * d
        x = torch.randn((M, width + stride), generator=g, device="cuda") * torch.exp2(torch.randn((M, 1), generator=g, device="cuda") * 2)
        self.x = (x if kind == "float" else x.to(torch.bfloat16))[:, :width]
        w = lambda c: 1 + 0.3 * torch.randn(d, generator=g, device="cuda") if c in norm else None
        self.wq, self.wk = w("q"), w("k")
        self.freq = (1e4 ** (-2 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)).float() if rot else None
        self.pos = torch.randint(0, pos_hi + 1, (M,), generator=g, device="cuda", dtype=torch.int32)
        self.hq, self.hkv, self.d, self.rot, self.inter, self.scale, self.eps = hq, hkv, d, rot, interleaved, scale, eps
        self.form = w12.QKVForm(hq, hkv, d, q_norm=self.wq, k_norm=self.wk, eps=eps, inv_freq=self.freq, interleaved=interleaved,
                                rot_scale=scale)

    def exact(self):
        """(values, sizes of a column and its partner) of q, k, v."""
        x = self.x.double().unflatten(1, (-1, self.d))
        out = []
        for y, w in zip(x.split([self.hq, self.hkv, self.hkv], 1), (self.wq, self.wk, None)):
            size = y.abs()
            if len(out) < 2:
                if w is not None:
                    y = y / (y.square().mean(2, keepdim=True) + self.eps).sqrt() * w.double()
                size = y.abs()
                if self.rot:
                    h = self.rot // 2
                    a = slice(0, self.rot, 2) if self.inter else slice(0, h)
                    b = slice(1, self.rot, 2) if self.inter else slice(h, self.rot)
                    t = self.pos.double()[:, None, None] * self.freq.double()
                    z, s = y.clone(), size.clone()
                    z[..., a] = self.scale * (y[..., a] * t.cos() - y[..., b] * t.sin())
                    z[..., b] = self.scale * (y[..., b] * t.cos() + y[..., a] * t.sin())
                    s[..., a] = s[..., b] = abs(self.scale) * (size[..., a] + size[..., b])
                    y, size = z, s
            out.append((y, size))
        return out


def close(got, want, rows=None):
    for g, (y, size) in zip(got, want):
        if rows is not None:
            g, y, size = g[rows], y[rows], size[rows]
        err = (g.double() - y).abs()
        bound = 2.0 ** -8 * y.abs() + 2.0 ** -18 * size
        assert bool((err <= bound).all()), f"worst {float((err / bound.clamp(min=1e-30)).max())} of the bound"


FORMS = [  # hq, hkv, d, rot
    (40, 8, 128, 128), (1, 1, 8, 8), (3, 1, 64, 64), (7, 1, 96, 64), (24, 4, 256, 64), (6, 2, 256, 256), (5, 5, 72, 32),
    (2, 1, 16, 0), (9, 3, 128, 8), (33, 1, 136, 136)]


@pytest.mark.parametrize("hq,hkv,d,rot", FORMS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", ["float", "bf16"])
def test_rope_forms(w12, hq, hkv, d, rot, inter, kind):
    r = Rows(w12, d + rot, 5, hq, hkv, d, rot, interleaved=inter, kind=kind)
    out = w12.qkv_rope(r.x, r.form, r.pos)
    assert [t.dtype for t in out] == [torch.bfloat16] * 3
    close(out, r.exact())


@pytest.mark.parametrize("M", [1, 2, 151, 1217, 4099])
@pytest.mark.parametrize("norm", ["", "q", "k", "qk"])
def test_rope_rows_and_norms(w12, M, norm):
    r = Rows(w12, M, M, 6, 2, 128, 128, norm=norm, kind="float" if M % 2 else "bf16", stride=8 * (M % 3), scale=1.25)
    close(w12.qkv_rope(r.x, r.form, r.pos), r.exact())


def test_rope_far_positions(w12):
    r = Rows(w12, 3, 64, 2, 1, 128, 128, pos_hi=2 ** 31 - 2)
    r.pos[:2] = torch.tensor([2 ** 31 - 1, 0], dtype=torch.int32)
    close(w12.qkv_rope(r.x, r.form, r.pos), r.exact())


def test_rope_zero_rows_and_small_values(w12):
    r = Rows(w12, 4, 4, 2, 2, 64, 32, eps=0.0)
    r.x[0] = 1e-12                                      # squares of 1e-24 in float
    r.x[1] *= 1e-3
    close(w12.qkv_rope(r.x, r.form, r.pos), r.exact())
    r = Rows(w12, 4, 2, 2, 2, 64, 32)
    r.x[0] = 0.0
    out = w12.qkv_rope(r.x, r.form, r.pos)
    assert all(bool((t[0] == 0).all()) for t in out)
    close(out, r.exact())


@pytest.mark.parametrize("inter", [False, True])
def test_rope_padding_and_parts_of_one_array(w12, inter):
    r = Rows(w12, 5, 37, 6, 2, 128, 64, interleaved=inter)
    r.pos[::5] = -1
    r.pos[36] = -2 ** 31
    live = r.pos >= 0
    one = torch.full((37, 10 * 128 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k, v = (one[:, a:b].unflatten(1, (-1, 128)) for a, b in ((0, 768), (768, 1024), (1024, 1280)))
    got = w12.qkv_rope(r.x, r.form, r.pos, q=q, k=k, v=v)
    assert got[0] is q
    close(got, r.exact(), live)
    assert bool((one[~live] == 7).all()) and bool((one[:, 1280:] == 7).all())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", [(40, 8, 128, 128), (5, 1, 72, 32)])
def test_rope_in_place(w12, inter, hq, hkv, d, rot):
    r = Rows(w12, 6, 300, hq, hkv, d, rot, interleaved=inter, kind="bf16")
    want, apart = r.exact(), w12.qkv_rope(r.x, r.form, r.pos)
    cut = [0, hq * d, (hq + hkv) * d, (hq + 2 * hkv) * d]
    q, k, v = (r.x[:, a:b].unflatten(1, (-1, d)) for a, b in zip(cut, cut[1:]))
    w12.qkv_rope(r.x, r.form, r.pos, q=q, k=k, v=v)
    close((q, k, v), want)
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), apart))


def test_rope_refusals(w12):
    r = Rows(w12, 7, 4, 4, 2, 64, 64, kind="bf16")
    q, k, v = w12.qkv_rope(r.x, r.form, r.pos)
    for kw in (dict(q=k), dict(k=v[:3]), dict(v=q)):
        with pytest.raises(ValueError):
            w12.qkv_rope(r.x, r.form, r.pos, **kw)
    with pytest.raises(w12.W12Error):
        w12.qkv_rope(r.x, r.form, r.pos, k=v, v=v)
    with pytest.raises(w12.W12Error):                   # k in q's place
        w12.qkv_rope(r.x, r.form, r.pos, k=r.x[:, :128].unflatten(1, (2, 64)))
    with pytest.raises(ValueError):
        w12.qkv_rope(r.x, r.form, r.pos[:3])
    with pytest.raises(ValueError):
        w12.qkv_rope(r.x[:, :-8], r.form, r.pos)
    with pytest.raises(TypeError):
        w12.qkv_rope(r.x.half(), r.form, r.pos)
    with pytest.raises(ValueError):
        w12.qkv_rope(r.x, r.form, r.pos.long())


def test_rope_graph_and_stream(w12):
    r = Rows(w12, 8, 33, 6, 2, 128, 128)
    want = w12.qkv_rope(r.x, r.form, r.pos)
    out = [torch.zeros_like(t) for t in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = w12.qkv_rope(r.x, r.form, r.pos, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w12.qkv_rope(r.x, r.form, r.pos, *out)
    r.x.mul_(3.0)
    r.pos.add_(11)
    g.replay()
    torch.cuda.synchronize()
    close(out, r.exact())


# ---------------------------------------------------------------- into the cache

@pytest.mark.parametrize("block,layout", [(16, "nhd"), (1, "nhd"), (24, "hnd"), (7, "nhd"), (64, "hnd")])
@pytest.mark.parametrize("kind,inter", [("float", False), ("bf16", True)])
@pytest.mark.parametrize("rows", [False, True])
def test_append(w12, block, layout, kind, inter, rows):
    M, hkv, d = 41, 2, 128
    r = Rows(w12, block, M, 6, hkv, d, 128, interleaved=inter, kind=kind)
    blocks = -(-M // block) + 3
    shape = (3, blocks, block, hkv, d) if layout == "nhd" else (3, blocks, hkv, block, d)
    kc, vc = [torch.full(shape, 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    if layout == "hnd":
        kc, vc = kc.transpose(2, 3), vc.transpose(2, 3)
    rng = np.random.default_rng(block)
    slot = torch.from_numpy(rng.permutation(blocks * block)[:M]).cuda()
    slot[3] = -1                                        # no slot: its rows are written all the same
    r.pos[9] = -1                                       # padding, with a slot that must stay
    q, k, v, status = w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc, vc), slot, layer=1, rows=rows)
    live = r.pos >= 0
    want = r.exact()
    close((q,), want[:1], live)
    assert int(status) == 0 and (k is None) == (not rows) and (v is None) == (not rows)
    if rows:
        close((k, v), want[1:], live)
    put = live & (slot >= 0)
    for c, (y, size) in zip((kc, vc), want[1:]):
        flat = c[1].reshape(-1, hkv, d)
        close((flat[slot[put]],), [(y[put], size[put])])
        other = torch.ones(blocks * block, dtype=torch.bool, device="cuda")
        other[slot[put]] = False
        assert bool((flat[other] == 5).all()) and bool((c[0] == 5).all()) and bool((c[2] == 5).all())


def test_append_equals_rope_and_write(w12):
    """What kv_write later makes of qkv_rope's rows, bit for bit."""
    r = Rows(w12, 1, 100, 40, 8, 128, 128)
    caches = [[torch.zeros((9, 16, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    slot = torch.randperm(144, device="cuda")[:100]
    q, k, v = w12.qkv_rope(r.x, r.form, r.pos)
    w12.kv_write(w12.KVCache(*caches[0]), k, v, slot)
    q2, _, _, _ = w12.kv_append(r.x, r.form, r.pos, w12.KVCache(*caches[1]), slot)
    assert torch.equal(q, q2) and all(torch.equal(a, b) for a, b in zip(*caches))


def test_append_bad_slots(w12):
    r = Rows(w12, 2, 6, 2, 1, 64, 64)
    kc, vc = [torch.full((4, 16, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slot = torch.tensor([64, -2, 2 ** 40, -2 ** 63, 3, -1], dtype=torch.int64, device="cuda")
    q, k, v, status = w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc, vc), slot, rows=True)
    assert int(status) == 1
    close((q, k, v), r.exact())
    flat = kc.reshape(64, 64)
    assert bool((flat[[i for i in range(64) if i != 3]] == 5).all()) and not bool((flat[3] == 5).all())
    with pytest.raises(ValueError):
        w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc, vc), slot[:5])
    with pytest.raises(ValueError):
        w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc.view(4, 8, 2, 64), vc.view(4, 8, 2, 64)), slot)
    with pytest.raises(w12.W12Error):
        w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc, vc), slot, layer=1)
    with pytest.raises(w12.W12Error):                   # rows in the cache
        w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc, vc), slot, k=kc.view(64, 1, 64)[:6])


def test_append_far_slots(w12):
    """Places in the cache past 2^31 elements."""
    kc, vc = [torch.empty((2, 5 << 20, 1, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    r = Rows(w12, 3, 3, 4, 4, 128, 128)
    slot = torch.tensor([(5 << 20) - 1, 0, (4 << 20) + 77], dtype=torch.int64, device="cuda")
    _, _, _, status = w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc, vc), slot, layer=1)
    assert int(status) == 0
    close((kc[1].flatten(0, 1)[slot], vc[1].flatten(0, 1)[slot]), r.exact()[1:])


# ---------------------------------------------------------------- positions

def positions(lens, counts, parents, rows):
    out = np.full(rows, -1, np.int64)
    at = 0
    for r, n in enumerate(counts):
        depth = []
        for i in range(n):
            depth.append(i if parents is None else 0 if i == 0 else depth[parents[at + i]] + 1)
        out[at:at + n] = lens[r] + np.array(depth, np.int64)
        at += n
    return out


@pytest.mark.parametrize("counts", [[1], [8, 1, 0, 33], [256] * 3, [1000, 24], [4096], [0, 5], [1] * 700])
@pytest.mark.parametrize("shape", ["tree", "chain", "star", "none"])
@pytest.mark.parametrize("pad", [0, 9])
def test_positions(w12, counts, shape, pad):
    rng = np.random.default_rng(len(counts))
    lens = rng.integers(0, 100000, len(counts))
    up = {"tree": lambda i: int(rng.integers(max(0, i - 5), i)), "chain": lambda i: i - 1, "star": lambda i: 0}.get(shape)
    parents = None if up is None else [p for n in counts for p in ([-1] + [up(i) for i in range(1, n)] if n else [])]
    rows = sum(counts) + pad
    given = None if parents is None else i32(parents + [0] * pad)
    pos, status = w12.tree_positions(i32(lens), given, i32(np.concatenate([[0], np.cumsum(counts)])), rows=rows)
    assert int(status) == 0
    assert np.array_equal(pos.cpu().numpy(), positions(lens, counts, parents, rows))


def test_positions_of_one_request(w12):
    assert w12.tree_positions(i32([7]), i32([-1, 0, 0, 2]))[0].tolist() == [7, 8, 8, 9]
    assert w12.tree_positions(i32([7]), rows=3)[0].tolist() == [7, 8, 9]
    n = 300001
    assert torch.equal(w12.tree_positions(i32([5]), rows=n)[0].long(), torch.arange(5, n + 5, device="cuda"))


@pytest.mark.parametrize("shape", ["tree", "none"])
def test_positions_out_of_range(w12, shape):
    tree = [-1, 0, 0, -1, 0, -1, 0, 1, -1, 0]
    lens, off = [3, -1, 2 ** 31 - 3, 9], [0, 3, 5, 8, 10]   # a negative length; positions up to 2^31 - 1
    pos, status = w12.tree_positions(i32(lens), i32(tree) if shape == "tree" else None, i32(off), rows=10)
    assert int(status) == 1
    assert pos.tolist() == [3, 4, 4 if shape == "tree" else 5, -1, -1, -1, -1, -1, 9, 10]
    for bad in ([0, 3, 2, 8, 10], [0, 3, 5, 8, 11], [-1, 3, 5, 8, 10]):
        _, status = w12.tree_positions(i32([1] * 4), i32(tree) if shape == "tree" else None, i32(bad), rows=10)
        assert int(status) == 1
    if shape == "tree":
        for p in ([0, 0, 0], [-1, 1, 0], [-1, 0, -1], [-1, 5, 0]):
            pos, status = w12.tree_positions(i32([1, 4]), i32(p + [-1, 0]), i32([0, 3, 5]))
            assert int(status) == 1 and pos.tolist() == [-1, -1, -1, 4, 5]
        pos, status = w12.tree_positions(i32([1]), i32([-1] + list(range(4096))))   # 4097 nodes
        assert int(status) == 1 and bool((pos == -1).all())
