"""tree_attn against a plain 64-bit implementation.

Tolerance.  Products of bf16 values are exact in float and scores stay near 2^5, so scores
and sums carry errors of 2^-18 or less.  What is left are the roundings to bf16 (2^-9
relative each): of the probabilities, on the numerator only, at most 2^-9 sum p|v|, and of the
output, 2^-9 |out|.  With the float errors counted as another 2^-9 sum p|v|:
    |out - ref| <= 2^-9 (1 + 2^-7) |ref| + 2^-8 sum p|v|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests._gpu_util import f32_of_bf16, to_dev16, to_np16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lossless_bit_weights_gb300 as m
    m.lib()
    return m


def bf16(a):
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def tree(rng, n, kind="bushy"):
    if n == 0:
        return []
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    return [-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)]


def ancestors(parent):
    may = np.zeros((len(parent), len(parent)), bool)
    for i in range(len(parent)):
        p = i
        while p >= 0:
            may[i, p] = True
            p = parent[p]
    return may


class Problem:
    """Inputs as bf16 bits on the host and, in the asked layout, on the device."""

    def __init__(self, seed, lens, counts, hkv, group, d, block, layout="nhd", kind="bushy", spare=2, layers=1,
                 q_scale=2.0):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.hkv, self.group, self.d, self.block = lens, counts, hkv, group, d, block
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        M, R, hq = int(self.off[-1]), len(lens), hkv * group
        self.parents = [tree(rng, n, kind) for n in counts]
        need = [-(-n // block) for n in lens]
        blocks = sum(need) + spare
        ids = rng.permutation(blocks)
        self.table = np.full((R, max(1, max(need))), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.layers, self.layer = layers, layers - 1
        # everything the call must not read is NaN: other layers, unused blocks, tokens past a length
        self.kc = np.full((layers, blocks, block, hkv, d), 0x7FC0, np.uint16)
        self.vc = self.kc.copy()
        for r, n in enumerate(lens):
            for j in range(need[r]):
                m = min(block, n - j * block)
                for c in (self.kc, self.vc):
                    c[self.layer, self.table[r, j], :m] = bf16(rng.standard_normal((m, hkv, d)))
        self.q = bf16(rng.standard_normal((M, hq, d)) * q_scale)
        self.k = bf16(rng.standard_normal((M, hkv, d)))
        self.v = bf16(rng.standard_normal((M, hkv, d)))
        self.layout = layout

    def args(self, w12, strided=True):
        kc, vc = to_dev16(self.kc), to_dev16(self.vc)
        if self.layout == "hnd":  # heads outside tokens in memory
            kc, vc = (t.transpose(2, 3).contiguous().transpose(2, 3) for t in (kc, vc))
        elif self.layout == "halves":  # K and V of a block side by side
            both = torch.stack([kc, vc], 2)
            kc, vc = both[:, :, 0], both[:, :, 1]
        M = int(self.off[-1])
        if strided:
            flat = np.concatenate([x.reshape(M, -1) for x in (self.q, self.k, self.v)], 1)
            flat = to_dev16(flat)
            a, b = self.q[0].size, self.q[0].size + self.k[0].size
            q = flat[:, :a].unflatten(1, self.q.shape[1:])
            k = flat[:, a:b].unflatten(1, self.k.shape[1:])
            v = flat[:, b:].unflatten(1, self.k.shape[1:])
        else:
            q, k, v = to_dev16(self.q), to_dev16(self.k), to_dev16(self.v)
        parent = i32(np.concatenate([np.asarray(p, np.int32) for p in self.parents]) if M else [])
        return (q, k, v, w12.KVCache(kc, vc), i32(self.table), i32(self.lens), parent, i32(self.off))

    def reference(self, r, scale=None):
        """(out, sum p|v|) of request r in float64."""
        scale = self.d ** -0.5 if scale is None else scale
        n, m, o = self.lens[r], self.counts[r], int(self.off[r])
        ids = self.table[r, :-(-n // self.block)]
        f = lambda x: f32_of_bf16(x).astype(np.float64)
        K, V = (f(c[self.layer, ids].reshape(-1, self.hkv, self.d)[:n]) for c in (self.kc, self.vc))
        K, V = np.concatenate([K, f(self.k[o:o + m])]), np.concatenate([V, f(self.v[o:o + m])])
        may = np.concatenate([np.ones((m, n), bool), ancestors(self.parents[r])], 1)
        q = f(self.q[o:o + m])
        out, mag = np.zeros((m, self.hkv * self.group, self.d)), np.zeros((m, self.hkv * self.group, self.d))
        for h in range(self.hkv):
            rows = q[:, h * self.group:(h + 1) * self.group].reshape(-1, self.d)
            ok = np.repeat(may, self.group, 0)
            with np.errstate(invalid="ignore", over="ignore"):
                s = rows @ K[:, h].T * scale
                s = np.where(ok, s, -np.inf)
                p = np.where(ok, np.exp(s - s.max(1, keepdims=True)), 0.0)
                p /= p.sum(1, keepdims=True)
                # a token that a node does not attend to has no part in its sum, whatever it holds
                bad = ~np.isfinite(V[:, h]).all(1)
                o_ = p[:, ~bad] @ V[~bad, h]
                a_ = p[:, ~bad] @ np.abs(V[~bad, h])
                for j in np.flatnonzero(bad):
                    o_[ok[:, j]] += p[ok[:, j], j][:, None] * V[j, h]
            out[:, h * self.group:(h + 1) * self.group] = o_.reshape(m, self.group, self.d)
            mag[:, h * self.group:(h + 1) * self.group] = a_.reshape(m, self.group, self.d)
        return out, mag

    def check(self, out, requests=None, scale=None):
        got = f32_of_bf16(to_np16(out)).astype(np.float64)
        for r in range(len(self.lens)) if requests is None else requests:
            if not self.counts[r]:
                continue
            ref, mag = self.reference(r, scale)
            mine = got[self.off[r]:self.off[r + 1]]
            fin = np.isfinite(ref)
            assert np.array_equal(fin, np.isfinite(mine)), f"request {r}: finite in other places"
            assert np.array_equal(np.isnan(ref), np.isnan(mine)), f"request {r}: NaN in other places"
            tol = 2.0 ** -9 * (1 + 2.0 ** -7) * np.abs(ref) + 2.0 ** -8 * mag
            err = np.abs(mine[fin] - ref[fin])
            assert (err <= tol[fin]).all(), f"request {r}: {(err / tol[fin]).max():.3g} of the tolerance"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("length", [0, 1, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
def test_lengths(w12, d, length):
    p = Problem(length, [length], [5], 2, 3, d, 16)
    out, st = w12.tree_attn(*p.args(w12))
    p.check(out)
    assert int(st) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nodes", [1, 2, 16, 43, 64, 127, 128, 129, 200, 256])
@pytest.mark.parametrize("kind", ["bushy", "chain", "star"])
def test_trees(w12, d, nodes, kind):
    p = Problem(nodes, [300], [nodes], 2, 1, d, 32, kind=kind)
    out, st = w12.tree_attn(*p.args(w12))
    p.check(out)
    assert int(st) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hkv,group", [(1, 1), (3, 1), (1, 7), (8, 5), (2, 16), (1, 129)])
def test_heads(w12, d, hkv, group):
    p = Problem(hkv * group, [517, 40], [3, 9], hkv, group, d, 16)
    out, st = w12.tree_attn(*p.args(w12))
    p.check(out)
    assert int(st) == 0


@pytest.mark.parametrize("layout", ["nhd", "hnd", "halves"])
@pytest.mark.parametrize("block", [1, 3, 8, 16, 24, 100, 128, 300])
def test_blocks_and_layouts(w12, block, layout):
    for d in (64, 128, 256):
        p = Problem(block, [700, 1, 255], [6, 3, 11], 2, 2, d, block, layout, layers=2)
        args = p.args(w12)
        out, st = w12.tree_attn(*args, layer=1)
        p.check(out)
        assert int(st) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_uneven_requests_and_empty_ones(w12, d):
    lens = [0, 3000, 17, 0, 640, 1, 5000, 128, 0, 63]
    counts = [4, 1, 0, 0, 33, 70, 8, 0, 1, 2]
    p = Problem(3, lens, counts, 2, 5, d, 16)
    out, st = w12.tree_attn(*p.args(w12))
    p.check(out)
    assert int(st) == 0


def test_many_requests(w12):
    rng = np.random.default_rng(0)
    R = 700
    p = Problem(4, rng.integers(0, 90, R).tolist(), rng.integers(0, 4, R).tolist(), 1, 2, 64, 8)
    out, st = w12.tree_attn(*p.args(w12))
    p.check(out)
    assert int(st) == 0


@pytest.mark.parametrize("d,hkv,group,nodes", [(128, 1, 5, 16), (128, 2, 5, 64), (256, 1, 6, 32), (64, 1, 1, 1), (128, 1, 8, 1)])
def test_long_contexts(w12, d, hkv, group, nodes):
    p = Problem(9, [40001], [nodes], hkv, group, d, 64)
    args = p.args(w12)
    out, st = w12.tree_attn(*args)
    p.check(out)
    assert int(st) == 0
    again, _ = w12.tree_attn(*args)
    assert torch.equal(out, again)                       # the same bits on every call


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,counts", [([200] * 400, [1] * 400), ([1000, 40, 5000] * 40, [3, 60, 2] * 40),
                                         ([130] * 90, [40, 1, 70] * 30)])
def test_several_units_per_block(w12, d, lens, counts):
    """More work than blocks: each takes several heads and requests in turn, and parts of some."""
    p = Problem(len(lens), lens, counts, 2, 4, d, 16)
    args = p.args(w12)
    out, st = w12.tree_attn(*args)
    p.check(out)
    assert int(st) == 0
    again, _ = w12.tree_attn(*args)
    assert torch.equal(out, again)


def test_peaked_and_flat_scores(w12):
    """Scores from -100 to 100 (one key takes all) and all alike; a running maximum that keeps rising."""
    for q_scale in (0.0, 0.01, 8.0, 24.0):
        p = Problem(int(q_scale), [900], [12], 1, 4, 128, 16, q_scale=q_scale)
        out, _ = w12.tree_attn(*p.args(w12))
        p.check(out)
    p = Problem(5, [2000], [4], 1, 2, 128, 16)
    ramp = np.arange(2000) * 0.002
    one = np.ones((128,))
    for j, b in enumerate(p.table[0]):
        m = min(16, 2000 - j * 16)
        p.kc[0, b, :m, 0] = bf16(ramp[j * 16:j * 16 + m, None] * one)
    p.q[:] = bf16(np.ones_like(p.q, np.float32))
    out, _ = w12.tree_attn(*p.args(w12))
    p.check(out)


def test_a_given_scale(w12):
    p = Problem(6, [300], [7], 2, 2, 64, 16)
    out, _ = w12.tree_attn(*p.args(w12), scale=0.5)
    p.check(out, scale=0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [0x7F80, 0xFF80, 0x7FC0])
def test_what_a_node_does_not_attend_to_does_not_reach_it(w12, d, value):
    """Infinities and NaN in the K and V of nodes: only their descendants and themselves see them."""
    p = Problem(11, [150], [40], 2, 2, d, 16)
    for i in (7, 20, 39):
        p.v[i, 1, 3::9] = value
    out, _ = w12.tree_attn(*p.args(w12))
    p.check(out)
    p = Problem(12, [150], [40], 2, 2, d, 16)
    p.k[11, 0, 5] = 0x7FC0                                # a NaN score for node 11's descendants
    out, _ = w12.tree_attn(*p.args(w12))
    p.check(out)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_infinities_in_the_cache_reach_every_row(w12, d):
    p = Problem(13, [200], [9], 1, 2, d, 16)
    p.vc[0, p.table[0, 3], 2, 0, 5] = 0x7F80
    out, _ = w12.tree_attn(*p.args(w12))
    p.check(out)


def test_a_chain_is_causal_attention_and_one_node_is_decoding(w12):
    """A request's tokens in one pass of a chain, and one by one through kv_write and one-node
    passes: the same attention."""
    n, hkv, group, d, block = 37, 2, 3, 128, 16
    p = Problem(14, [0], [n], hkv, group, d, block, kind="chain")
    q, k, v, _, _, _, parent, off = p.args(w12)
    chain, _ = w12.tree_attn(q, k, v, w12.KVCache(*[torch.empty((3, block, hkv, d), dtype=torch.int16, device="cuda")
                                                    for _ in range(2)]), i32([[0]]), i32([0]), parent, off)
    p.check(chain)
    kc, vc = (torch.full((3, block, hkv, d), 0x7FC0, dtype=torch.int16, device="cuda") for _ in range(2))
    cache, table = w12.KVCache(kc, vc), i32([[2, 0, 1]])
    for t in range(n):
        one, _ = w12.tree_attn(q[t:t + 1], k[t:t + 1], v[t:t + 1], cache, table, i32([t]), i32([-1]), i32([0, 1]))
        a, b = (f32_of_bf16(to_np16(x)) for x in (one[0], chain[t]))
        assert np.abs(a - b).max() <= 2.0 ** -6 * np.abs(b).max()
        slot = torch.tensor([int(table[0, t // block]) * block + t % block], device="cuda")
        w12.kv_write(cache, k[t:t + 1], v[t:t + 1], slot)


def test_offsets_past_32_bits(w12):
    """A cache of more than 2^31 elements: the last blocks hold the request's tokens."""
    block, hkv, d = 64, 2, 128
    blocks = (1 << 31) // (block * hkv * d) + 50
    p = Problem(15, [500], [6], hkv, 2, d, block)
    kc, vc = (torch.empty((blocks, block, hkv, d), dtype=torch.int16, device="cuda") for _ in range(2))
    args = list(p.args(w12))
    used = p.kc.shape[1]
    for big, small in ((kc, p.kc), (vc, p.vc)):
        big[blocks - used:] = to_dev16(small[0])
    args[3] = w12.KVCache(kc, vc)
    args[4] = args[4] + (blocks - used)
    assert kc.stride(0) * (blocks - used) > 1 << 31
    out, st = w12.tree_attn(*args)
    p.check(out)
    assert int(st) == 0


def test_another_stream_and_one_workspace(w12):
    ws = w12.Workspace()
    small, big = Problem(16, [90], [2], 2, 2, 128, 16), Problem(17, [9000], [30], 2, 5, 128, 16)
    s = torch.cuda.Stream()
    for p in (small, big, small):
        args = p.args(w12)
        s.wait_stream(torch.cuda.current_stream())
        out, st = w12.tree_attn(*args, ws=ws, stream=s)
        s.synchronize()
        p.check(out)
    A = w12.encode(to_dev16(bf16(np.random.default_rng(0).standard_normal((512, 256)))))
    x = to_dev16(bf16(np.random.default_rng(1).standard_normal((4, 256))))
    first = w12.w12_gemm(x, A)
    w12.tree_attn(*big.args(w12), ws=ws)
    assert torch.equal(w12.w12_gemm(x, A, ws=ws), first)  # the GEMM's counters were left alone
    assert ws.status() == 0


def test_in_a_graph(w12):
    p = Problem(18, [3000, 5], [9, 3], 2, 5, 128, 16)
    args, ws = p.args(w12), w12.Workspace()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(args[0].shape, dtype=torch.int16, device="cuda")
    w12.tree_attn(*args, out=out, ws=ws, status=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w12.tree_attn(*args, out=out, ws=ws, status=st)
    out.zero_()
    args[5].copy_(i32([2900, 5]))                         # lengths are read on the device
    g.replay()
    p.lens = [2900, 5]
    p.check(out)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_out_of_range_requests_are_reported_and_left_alone(w12, d):
    lens, counts = [200, 300, 90, 500, 40], [5, 6, 4, 3, 2]

    def call(change):
        p = Problem(19, lens, counts, 2, 2, d, 16)
        args = list(p.args(w12))
        change(p, args)
        out = torch.full(args[0].shape, 0x1234, dtype=torch.int16, device="cuda")
        _, st = w12.tree_attn(*args, out=out)
        return p, out, int(st)

    def bad(args, i, at, value):
        args[i] = args[i].clone()
        args[i][at] = value

    cases = [(1, 1, lambda p, a: bad(a, 6, int(p.off[1]), 0)),            # the root has a parent
             (1, 1, lambda p, a: bad(a, 6, int(p.off[1]) + 3, 3)),        # a node is its own parent
             (1, 1, lambda p, a: bad(a, 6, int(p.off[1]) + 3, 77)),
             (1, 1, lambda p, a: bad(a, 5, 1, -1)),                       # lengths
             (1, 1, lambda p, a: bad(a, 5, 1, p.table.shape[1] * 16 + 1)),
             (2, 1, lambda p, a: bad(a, 4, (1, 5), p.kc.shape[1])),       # blocks outside the cache
             (2, 1, lambda p, a: bad(a, 4, (1, 18), -5))]
    for want, r, change in cases:
        p, out, st = call(change)
        assert st == want
        p.check(out, [i for i in range(5) if i != r])
        assert (out[p.off[r]:p.off[r + 1]] == 0x1234).all()


@pytest.mark.parametrize("d,block", [(64, 16), (128, 16), (128, 24), (256, 64)])
def test_a_wait_that_runs_out_is_reported(w12, d, block):
    """Waits bounded far below a tile's latency: every role gives up, nothing stays in flight, the
    call ends and reports it, and the next call on the same workspace gives the full result."""
    p = Problem(23, [3000, 40, 700], [30, 5, 60], 2, 3, d, block)
    args, ws = p.args(w12), w12.Workspace()
    first, st = w12.tree_attn(*args, ws=ws)
    assert int(st) == 0
    w12.tree_attn_set_wait_limit(64)
    try:
        _, st = w12.tree_attn(*args, ws=ws)
        torch.cuda.synchronize()
    finally:
        w12.tree_attn_set_wait_limit(0)
    assert int(st) & 4
    again, st = w12.tree_attn(*args, ws=ws)
    assert int(st) == 0 and torch.equal(first, again)
    p.check(again)


def test_too_many_nodes_are_reported(w12):
    p = Problem(20, [100, 30], [257, 3], 1, 1, 64, 16)
    out, st = w12.tree_attn(*p.args(w12))
    assert int(st) == 1
    p.check(out, [1])


def test_offsets_out_of_range_are_reported(w12):
    p = Problem(21, [100, 30, 60], [5, 3, 2], 1, 1, 64, 16)
    args = list(p.args(w12))
    args[7] = i32([0, 5, 8, 4000])
    out, st = w12.tree_attn(*args)
    assert int(st) == 1
    p.check(out, [0, 1])


def test_out_must_not_overlap_its_inputs(w12):
    p = Problem(22, [100], [5], 2, 2, 64, 16)
    q, k, v, cache, table, lens, parent, off = p.args(w12)
    both = torch.zeros((2 * q.shape[0],) + tuple(q.shape[1:]), dtype=q.dtype, device="cuda")
    n = q.shape[0]
    both[:n] = q
    for out in (both[:n], both[1:n + 1]):
        with pytest.raises(w12.W12Error, match="overlap") as e:
            w12.tree_attn(both[:n], k, v, cache, table, lens, parent, off, out=out)
        assert e.value.status == 1
    out, st = w12.tree_attn(both[:n], k, v, cache, table, lens, parent, off, out=both[n:])
    assert int(st) == 0
    p.check(out)


def test_refusals(w12):
    p = Problem(22, [100], [5], 2, 2, 64, 16)
    q, k, v, cache, table, lens, parent, off = p.args(w12)
    call = w12.tree_attn
    with pytest.raises(TypeError):
        call(q.float(), k, v, cache, table, lens, parent, off)
    with pytest.raises(ValueError):
        call(q, k[:, :1], v, cache, table, lens, parent, off)
    with pytest.raises(ValueError):
        call(q, k, v, cache, table.long(), lens, parent, off)
    with pytest.raises(ValueError):
        call(q, k, v, cache, table, lens, parent[:4], off)
    with pytest.raises(ValueError):
        call(q, k, v, cache, table, lens, parent, i32([0, 2, 5]))
    with pytest.raises(ValueError):
        call(q, k, v, cache, torch.cat([table, table]), i32([100, 100]), parent)
    with pytest.raises(ValueError):
        call(q.cpu(), k, v, cache, table, lens, parent, off)
    with pytest.raises(ValueError):
        call(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cache, table, lens, parent, off)
    for kw, status in (({"layer": 1}, 2), ({"scale": float("nan")}, 1), ({"scale": -1.0}, 1)):
        with pytest.raises(w12.W12Error) as e:
            call(q, k, v, cache, table, lens, parent, off, **kw)
        assert e.value.status == status
    with pytest.raises(w12.W12Error):                     # three query heads on two
        call(q[:, :3].contiguous(), k, v, cache, table, lens, parent, off)
    with pytest.raises(ValueError):
        w12.KVCache(cache.k, cache.v[:, :1])
    odd = torch.empty((4, 16, 2, 96), dtype=torch.int16, device="cuda")
    with pytest.raises(w12.W12Error) as e:                # head_dim 96
        call(torch.zeros((5, 4, 96), dtype=torch.int16, device="cuda"), *[torch.zeros((5, 2, 96), dtype=torch.int16, device="cuda")] * 2,
             w12.KVCache(odd, odd), table, lens, parent, off)
    assert e.value.status == 2


@pytest.mark.parametrize("d,block", [(64, 16), (128, 32), (256, 64), (128, 24)])
def test_a_bad_block_anywhere_in_a_long_request(w12, d, block):
    """The request is split among many blocks of the grid, whose parts end in tiles of cached tokens: each of
    them has to tell what it met before its results are used."""
    lens, counts = [90, 20000, 40], [3, 4, 2]
    p = Problem(24, lens, counts, 2, 2, d, block)
    args, ws = list(p.args(w12)), w12.Workspace()
    good, last = args[4], -(-lens[1] // block) - 1
    rng = np.random.default_rng(d)
    for at in [0, 1, last - 1, last] + rng.integers(0, last, 60).tolist():
        for value in (-1, p.kc.shape[1], 2 ** 31 - 1):
            args[4] = good.clone()
            args[4][1, at] = value
            out = torch.full(args[0].shape, 0x1234, dtype=torch.int16, device="cuda")
            _, st = w12.tree_attn(*args, out=out, ws=ws)
            assert int(st) == 2, (at, value)
            assert (out[p.off[1]:p.off[2]] == 0x1234).all(), (at, value)
    p.check(out, [0, 2])
    args[4] = good
    out, st = w12.tree_attn(*args, ws=ws)
    assert int(st) == 0
    p.check(out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_req", [32, 33, 460])
def test_long_requests_beyond_a_warp_s_schedule(w12, d, n_req):
    """Above 32 requests the schedule's sums stand in the ring, whose first tiles land there by boxes."""
    lens = [512 if r % 7 else 2000 for r in range(n_req)]
    p = Problem(n_req, lens, [1 + r % 3 for r in range(n_req)], 1, 2, d, 64)
    args, ws = p.args(w12), w12.Workspace()
    out, st = w12.tree_attn(*args, ws=ws)
    p.check(out)
    assert int(st) == 0
    for _ in range(20):
        again, _ = w12.tree_attn(*args, ws=ws)
        assert torch.equal(out, again)


def test_one_workspace_on_two_streams_at_once(w12):
    """Calls on streams that do not wait for one another, over and over: each gives what it gives alone."""
    ws = w12.Workspace()
    ps = [Problem(25, [9000, 400], [30, 4], 2, 5, 128, 16), Problem(26, [7000], [16], 2, 5, 128, 16)]
    args = [p.args(w12) for p in ps]
    want = [w12.tree_attn(*a)[0] for a in args]
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [[torch.empty_like(x) for _ in range(40)] for x in want]
    status = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in ps]
    torch.cuda.synchronize()
    for i in range(40):
        for s, a, o, st in zip(streams, args, outs, status):
            w12.tree_attn(*a, out=o[i], ws=ws, status=st, stream=s)
    torch.cuda.synchronize()
    for p, x, o, st in zip(ps, want, outs, status):
        p.check(x)
        assert int(st) == 0 and all(torch.equal(x, y) for y in o)


def test_a_graph_after_a_larger_call(w12):
    """A capture on a stream that has called before, then a larger call on that stream: replays still find
    their buffer, and nothing else is found changed by them."""
    p, big = Problem(27, [9000, 5], [9, 3], 2, 5, 128, 16), Problem(28, [9000], [200], 2, 8, 128, 16)
    args, ws, s = p.args(w12), w12.Workspace(), torch.cuda.Stream()
    st, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(args[0], memory_format=torch.contiguous_format)
    torch.cuda.synchronize()
    w12.tree_attn(*args, out=out, ws=ws, status=st, stream=s)
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w12.tree_attn(*args, out=out, ws=ws, status=st)
    x, _ = w12.tree_attn(*big.args(w12), ws=ws, stream=s)
    torch.cuda.synchronize()
    big.check(x)
    with torch.cuda.stream(s):
        fresh = [torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]  # where a freed buffer stood
    torch.cuda.synchronize()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(out, want)
    assert all((t == 7).all() for t in fresh)
